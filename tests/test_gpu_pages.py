"""Pages of paged caches on the GPU: steps of a block table and compaction, against a
plain walk over Python lists."""

import random

import pytest
import torch

from gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dkv():
    require_cuda()
    import decode_attention_paged_kv_gb300 as m
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_caches(dkv, kind, nb, table, N, H=2, d=64, seed=0):
    """(cache objects, [tensors whose first dimension counts blocks])."""
    gen = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    if kind == "kv16":
        p = [r(nb, H, 16, d).bfloat16() for _ in "KV"]
        return [dkv.PagedCache(x, table, N) for x in p], p
    if kind == "kv_one":  # K and V in one tensor, a block's halves
        both = r(nb, 2, H, 16, d).half()
        return [dkv.PagedCache(both[:, i], table, N) for i in (0, 1)], [both]
    if kind.startswith("latent"):
        p = r(nb, int(kind[6:]), 320).bfloat16()
        return [dkv.LatentCache(p, table, N)], [p]
    c = [r(nb, H, 16, d).to(torch.float8_e4m3fn) for _ in "KV"]
    s = [r(nb, H).abs() for _ in "KV"]
    return ([dkv.Fp8PagedCache(c[i], s[i], table, N) for i in (0, 1)],
            [c[0].view(torch.uint8), s[0], c[1].view(torch.uint8), s[1]])


def fork_plain(table, refs, lens, parents, new, S):
    """The step on lists: (table, refs, [(from, to)]) or None if it does not fit."""
    B, P = len(table), len(table[0])
    nb = len(refs)
    if any(not -1 <= p < B for p in parents) or any(n < 0 for n in new):
        return None
    free = iter([i for i in range(nb) if refs[i] == 0])
    out, copies = [], []
    for b, p in enumerate(parents):
        kept = lens[p] if p >= 0 else 0
        if kept < 0 or kept + new[b] > P * S:
            return None
        row = list(table[p][:-(-kept // S)]) if p >= 0 else []
        if any(not 0 <= e < nb for e in row):
            return None
        if kept % S and (parents.index(p) != b or refs[row[-1]] > 1):
            to = next(free, None)
            if to is None:
                return None
            copies.append((row[-1], to))
            row[-1] = to
        while len(row) * S < kept + new[b]:
            to = next(free, None)
            if to is None:
                return None
            row.append(to)
        out.append(row + [-1] * (P - len(row)))
    refs = list(refs)
    for old, now in zip(table, out):
        for e in old:
            if 0 <= e < nb:
                refs[e] -= 1
        for e in now:
            if e >= 0:
                refs[e] += 1
    return out, refs, copies


def run_fork(dkv, caches, tensors, table, refs, lens, parents, new, S, ws):
    """One call and its check; returns the plain form's result (None: refused)."""
    t0, r0 = table.tolist(), refs.tolist()
    before = [x.clone() for x in tensors]
    dkv.kv_pages_fork(caches, refs, ints(lens), parents=None if parents is None else ints(parents),
                      new_lens=None if new is None else ints(new), workspace=ws)
    B = len(t0)
    want = fork_plain(t0, r0, lens, list(range(B)) if parents is None else parents,
                      [0] * B if new is None else new, S)
    assert dkv.read_device_status(ws) == (0 if want else 9)
    if want is None:
        assert table.tolist() == t0 and refs.tolist() == r0
        for x, y in zip(tensors, before):
            assert torch.equal(x, y)
        return None
    assert table.tolist() == want[0] and refs.tolist() == want[1]
    for x, y in zip(tensors, before):
        for src, dst in want[2]:
            y[dst] = y[src].clone()
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    return want


KINDS = ["kv16", "kv_one", "fp8", "latent16", "latent32", "latent64"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,P,nb,seed", [(1, 1, 3, 0), (4, 5, 40, 1), (9, 3, 24, 2), (33, 40, 700, 3),
                                         (130, 7, 5000, 4)])
def test_fork_steps(dkv, kind, B, P, nb, seed):
    # a run of random steps: rows continue, fork, end, begin and grow; some do not fit
    rng = random.Random(f"{kind}{seed}")
    S = int(kind[6:]) if kind.startswith("latent") else 16
    wide = torch.full((B, P + 3), -1, dtype=torch.int32, device="cuda")
    table = wide[:, :P]
    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    held = rng.sample(range(nb), nb // 10)
    refs[held] = 1
    caches, tensors = make_caches(dkv, kind, nb, table, P * S, H=rng.choice([1, 2, 3]), seed=seed)
    ws = torch.zeros(dkv.pages_workspace_bytes(B, P, nb), dtype=torch.uint8, device="cuda")
    lens = [0] * B
    for step in range(8):
        parents = [rng.choice([b, b, rng.randrange(B), -1]) for b in range(B)]
        room = [P * S - (lens[p] if p >= 0 else 0) for p in parents]
        new = [rng.choice([0, 1, 1, rng.randint(0, max(0, r))]) if r > 0 else 0 for r in room]
        if step % 3 == 2 and P * S < 1000:
            new = [rng.choice([0, r]) for r in room]
        want = run_fork(dkv, caches, tensors, table, refs, lens, parents, new, S, ws)
        if want:
            lens = [(lens[p] if p >= 0 else 0) + n for p, n in zip(parents, new)]
            # some sequences drop tokens again, as refused drafts do
            lens = [max(0, n - rng.choice([0, 0, 0, 5, 40])) for n in lens]
        assert bool((wide[:, P:] == -1).all())
        assert int(refs.min()) >= 0


def test_fork_defaults(dkv):
    # no parents, no new tokens: rows keep their length, pages past it are released
    table = ints([[5, 2, 7, -1], [1, -1, -1, -1]])
    refs = ints([0, 1, 1, 0, 0, 1, 0, 1, 0, 0])
    caches, tensors = make_caches(dkv, "kv16", 10, table, 64)
    ws = torch.zeros(dkv.pages_workspace_bytes(2, 4, 10), dtype=torch.uint8, device="cuda")
    want = run_fork(dkv, caches, tensors, table, refs, [17, 0], None, None, 16, ws)
    assert want[0] == [[5, 2, -1, -1], [-1] * 4]
    assert refs.tolist() == [0, 0, 1, 0, 0, 1, 0, 0, 0, 0]


def test_fork_last_page_of_two_owners(dkv):
    # a last page that another entry holds too is copied even for its only child
    table = ints([[3, 4], [3, 4]])
    refs = ints([0, 0, 0, 2, 2, 0])
    caches, tensors = make_caches(dkv, "fp8", 6, table, 32, H=3)
    ws = torch.zeros(dkv.pages_workspace_bytes(2, 2, 6), dtype=torch.uint8, device="cuda")
    want = run_fork(dkv, caches, tensors, table, refs, [20, 32], [0, 1], [1, 0], 16, ws)
    assert want[0] == [[3, 0], [3, 4]] and want[2] == [(4, 0)]


@pytest.mark.parametrize("lens,parents,new", [
    ([20, 40], [0, 2], [0, 0]), ([20, 40], [-2, 1], [0, 0]), ([20, 40], [0, 1], [-1, 0]),
    ([20, 40], [0, 1], [0, 100]), ([-1, 40], [0, 1], [0, 0]), ([20, 49], [0, 1], [0, 0]),
    ([2 ** 31 - 1, 40], [0, 1], [2 ** 31 - 1, 0]), ([33, 40], [0, 1], [0, 0]),
    ([20, 40], [1, 1], [100, 100]), ([33, 40], [0, 1], [40, 8])])
def test_fork_refused(dkv, lens, parents, new):
    # row 0 holds two pages, row 1 three; ten blocks, three of them free
    table = ints([[0, 1, -1, -1, 99, -1, -1, -1], [2, 3, 4, -1, -1, -1, -1, -1]])
    refs = ints([1, 1, 1, 1, 1, 1, 1, 0, 0, 0])
    caches, tensors = make_caches(dkv, "kv16", 10, table, 8 * 16)
    ws = torch.zeros(dkv.pages_workspace_bytes(2, 8, 10), dtype=torch.uint8, device="cuda")
    assert run_fork(dkv, caches, tensors, table, refs, lens, parents, new, 16, ws) is None
    # the workspace serves the next call; stale lengths of rows that end do not matter
    assert run_fork(dkv, caches, tensors, table, refs, [-7, 40], [-1, 1], [1, 8], 16, ws)


@pytest.mark.parametrize("B", [5000, 16384])
def test_fork_many_rows(dkv, B):
    # more rows than the first kernel has threads (and than its shared memory holds without
    # asking for more), pools of more blocks than it scans at once
    P, nb = 2, 9000 + 5 * B
    table = torch.full((B, P), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    refs[:9000] = 1
    caches, tensors = make_caches(dkv, "latent16", nb, table, 32)
    ws = torch.zeros(dkv.pages_workspace_bytes(B, P, nb), dtype=torch.uint8, device="cuda")
    rng = random.Random(5)
    new = [rng.randint(0, 31) for _ in range(B)]
    assert run_fork(dkv, caches, tensors, table, refs, [0] * B, [-1] * B, new, 16, ws)
    parents = [rng.randrange(B) for _ in range(B)]
    assert run_fork(dkv, caches, tensors, table, refs, new, parents, [1] * B, 16, ws)


def test_fork_captured(dkv):
    B, P, nb = 6, 9, 90
    table = torch.full((B, P), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    caches, tensors = make_caches(dkv, "kv16", nb, table, P * 16)
    ws = torch.zeros(dkv.pages_workspace_bytes(B, P, nb), dtype=torch.uint8, device="cuda")
    lens, parents, new = ints([0] * B), ints([-1] * B), ints([40 + b for b in range(B)])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dkv.kv_pages_fork(caches, refs, lens, parents=parents, new_lens=new, workspace=ws)
    state = (table.tolist(), refs.tolist())
    rng = random.Random(1)
    for _ in range(6):
        g.replay()
        torch.cuda.synchronize()
        state = fork_plain(*state, lens.tolist(), parents.tolist(), new.tolist(), 16)[:2]
        assert (table.tolist(), refs.tolist()) == (state[0], state[1])
        par = parents.tolist()
        n = [(lens.tolist()[p] if p >= 0 else 0) + k for p, k in zip(par, new.tolist())]
        lens.copy_(ints(n))
        parents.copy_(ints([rng.randrange(B) for _ in range(B)]))
        new.fill_(1)
    assert dkv.read_device_status(ws) == 0


def compact_plain(table, refs):
    nb = len(refs)
    live = [i for i in range(nb) if refs[i] > 0]
    n = len(live)
    src = [i for i in live if i >= n]
    dst = [i for i in range(n) if refs[i] <= 0]
    to = {i: i for i in live} | dict(zip(src, dst))
    count = [0] * nb
    for i in live:
        count[to[i]] = refs[i]
    return ([[to.get(e, -1) for e in row] for row in table], count,
            [to.get(i, -1) for i in range(nb)], list(zip(src, dst)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nb,live,inplace", [(1, 1.0, True), (5, 0.0, False), (64, 0.5, True),
                                             (4097, 0.3, False), (9000, 0.9, True),
                                             (8192, 1.0, False), (4096, 0.001, True)])
def test_compact(dkv, kind, nb, live, inplace):
    rng = random.Random(f"{kind}{nb}")
    S = int(kind[6:]) if kind.startswith("latent") else 16
    B, P = 7, 11
    table = ints([[rng.choice([-1, rng.randrange(nb), rng.randrange(nb)]) for _ in range(P)]
                  for _ in range(B)])
    refs = ints([rng.randint(1, 3) if rng.random() < live else rng.choice([0, 0, -1])
                 for _ in range(nb)])
    table[0, 0] = nb + 5  # not a block
    caches, tensors = make_caches(dkv, kind, nb, table, P * S, H=rng.choice([1, 3]), seed=nb)
    want = compact_plain(table.tolist(), refs.tolist())
    before = [x.clone() for x in tensors]
    kept = (table.clone(), refs.clone())
    kw = {} if inplace else dict(refs_out=torch.full_like(refs, -9),
                                 block_table_out=torch.full_like(table, -9))
    ws = torch.zeros(dkv.pages_workspace_bytes(B, P, nb), dtype=torch.uint8, device="cuda")
    to = dkv.kv_pages_compact(caches, refs, workspace=ws, **kw)
    assert dkv.read_device_status(ws) == 0
    assert to.tolist() == want[2]
    got_t, got_r = kw.get("block_table_out", table), kw.get("refs_out", refs)
    assert got_t.tolist() == want[0] and got_r.tolist() == want[1]
    if not inplace:
        assert torch.equal(table, kept[0]) and torch.equal(refs, kept[1])
    for x, y in zip(tensors, before):
        for src, dst in want[3]:
            y[dst] = y[src].clone()
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_compact_without_tables_of_its_own_stride(dkv):
    # a table that is a view, renamed into another view
    wide, out = ints([[7, 3, 11, 12], [3, -1, 13, 14]]), ints([[0] * 6, [0] * 6])
    table = wide[:, :2]
    refs = ints([0, 0, 0, 2, 0, 0, 0, 1])
    caches, _ = make_caches(dkv, "kv16", 8, table, 32)
    to = dkv.kv_pages_compact(caches, refs, block_table_out=out[:, 2:4])
    assert to.tolist() == [-1, -1, -1, 0, -1, -1, -1, 1]
    assert out.tolist() == [[0, 0, 1, 0, 0, 0], [0, 0, 0, -1, 0, 0]]
    assert refs.tolist() == [2, 1, 0, 0, 0, 0, 0, 0]
    assert wide.tolist() == [[7, 3, 11, 12], [3, -1, 13, 14]]


@pytest.mark.parametrize("kind", ["fp8", "kv16"])
def test_beams_over_a_cache(dkv, kind):
    """Beams that fork, append and attend over paged caches, as each of them alone over a
    dense copy: bit for bit, whatever pages they share."""
    B, H, d, N, steps = 4, 2, 64, 160, 30
    P = N // 16
    nb = B * P + 1
    gen = torch.Generator("cuda").manual_seed(3)
    table = torch.full((B, P), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    eight = kind == "fp8"
    caches, _ = make_caches(dkv, kind, nb, table, N, H=H, d=d, seed=9)
    dense = [torch.zeros(B, H, N, d, device="cuda").bfloat16() for _ in "KV"]
    if eight:
        dense = [dkv.Fp8Cache(x.to(torch.float8_e4m3fn), torch.zeros(B, H, P, device="cuda"))
                 for x in dense]
    ws = torch.zeros(max(dkv.pages_workspace_bytes(B, P, nb),
                         dkv.workspace_bytes(B, 4, H, d, N, fp8=eight)), dtype=torch.uint8,
                     device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    rng = random.Random(2)
    for step in range(steps):
        parents = [rng.randrange(B) if step else -1 for _ in range(B)]
        T = 40 if step == 0 else rng.choice([1, 1, 4])
        n = ints([rng.randint(1, T) for _ in range(B)])
        par = ints(parents)
        dkv.kv_pages_fork(caches, refs, lens, parents=par, new_lens=n, workspace=ws)
        assert dkv.read_device_status(ws) == 0
        if step:
            lens = lens[par.long()]
            for c in dense:
                if not eight:
                    c.copy_(c[par.long()])
                    continue
                c.codes.view(torch.uint8).copy_(c.codes.view(torch.uint8)[par.long()])
                c.scale.copy_(c.scale[par.long()])
        lens = lens + n
        k, v = (torch.randn(B, T, H, d, generator=gen, device="cuda").bfloat16() for _ in "kv")
        q = torch.randn(B, 4, d, generator=gen, device="cuda").bfloat16()
        outs = []
        for K, V in (caches, dense):
            dkv.kv_append(k, v, K, V, seq_lens=lens, new_lens=n, workspace=ws)
            outs.append(dkv.decode_attn_full(q, K, V, seq_lens=lens, workspace=ws))
        assert dkv.read_device_status(ws) == 0
        assert torch.equal(outs[0], outs[1]), step
        if int(lens.max()) + 8 > N:
            break


@pytest.mark.parametrize("kind", ["fp8", "kv16"])
def test_beams_select_pages(dkv, kind):
    """Beams that fork, append and attend page-sparsely: page metadata goes by rows of the
    table, so the caller gathers it by the parents before it is brought up to date; then
    selections and outputs are those of metadata built anew, bit for bit."""
    B, H, d, N, top_k = 4, 2, 64, 320, 3
    P = N // 16
    nb = B * P + 1
    gen = torch.Generator("cuda").manual_seed(4)
    table = torch.full((B, P), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    caches, _ = make_caches(dkv, kind, nb, table, N, H=H, d=d, seed=10)
    K, V = caches
    ws = torch.zeros(max(dkv.pages_workspace_bytes(B, P, nb),
                         dkv.workspace_bytes(B, 4, H, d, N, top_k, fp8=kind == "fp8")),
                     dtype=torch.uint8, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    meta = tuple(torch.zeros(B, H, P, d, dtype=torch.bfloat16, device="cuda") for _ in "nx")
    rng = random.Random(5)
    moved = 0
    for step in range(20):
        parents = [rng.randrange(B) if step else -1 for _ in range(B)]
        T = 150 if step == 0 else rng.choice([1, 1, 5])
        n = ints([rng.randint(T // 2 + 1, T) for _ in range(B)])
        par = ints(parents)
        dkv.kv_pages_fork(caches, refs, lens, parents=par, new_lens=n, workspace=ws)
        if step:
            lens = lens[par.long()]
            for x in meta:
                x.copy_(x[par.long()])
        lens = lens + n
        k, v = (torch.randn(B, T, H, d, generator=gen, device="cuda").bfloat16() for _ in "kv")
        q = torch.randn(B, 4, d, generator=gen, device="cuda").bfloat16()
        dkv.kv_append(k, v, K, V, seq_lens=lens, new_lens=n, workspace=ws)
        dkv.kv_meta_append(K, meta, seq_lens=lens, new_tokens=T, new_lens=n)
        anew = dkv.kv_meta_build(K, seq_lens=lens)
        got, want = (dkv.decode_attn_select(q, K, V, m, top_k, return_selected=True, seq_lens=lens,
                                            workspace=ws) for m in (meta, anew))
        assert dkv.read_device_status(ws) == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), step
        for b in range(B):
            pages = (int(lens[b]) + 15) // 16
            assert all(torch.equal(x[b, :, :pages], y[b, :, :pages]) for x, y in zip(meta, anew))
        moved += sum(p != b for b, p in enumerate(parents))
    assert moved > 20
