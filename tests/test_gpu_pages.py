"""Copying, forking and compacting pages against their definitions (oracle.cache): tables, lengths, moves
and counts equal, pool contents equal bit for bit, untouched positions untouched."""

import numpy as np
import pytest
import torch

import oracle.cache as oc
import paged_split_kv_append_gb300 as nbx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def pools(num_pages, h, P, d, kind, seed, T=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (num_pages, h, P, d)
    if kind == "e4m3":
        out = [torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
               for _ in range(2)]
    else:
        out = [torch.randn(shape, generator=g, device=DEV).to(TYPES[kind]) for _ in range(2)]
    if T:
        out += [torch.randn((num_pages, h, P // T), generator=g, device=DEV) for _ in range(2)]
    return out


def moved(pools_, moves, T=0):
    """The pools after the moves, on the host side of the definition."""
    ref = [t.clone() for t in pools_]
    for s, d, n in moves:
        for t in ref[:2]:
            t[d, :, :n] = t[s, :, :n]
        for t in ref[2:]:
            t[d, :, : -(-n // T)] = t[s, :, : -(-n // T)]
    return ref


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def table_for(lens, P, width, seed, spread=1.5, reserve=0):
    g = np.random.default_rng(seed)
    need = [-(-n // P) + reserve if n else 0 for n in lens]
    num_pages = max(2, int(sum(need) * spread) + 1)
    ids = g.permutation(num_pages).astype(np.int32)
    t = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        k = min(k, width)
        t[b, :k] = ids[at:at + k]
        at += k
    return t, num_pages


SHAPES = [("bf16", 2, 16, 128, 0), ("f32", 1, 32, 64, 0), ("e4m3", 3, 64, 256, 0), ("e4m3", 2, 64, 64, 32),
          ("bf16", 4, 64, 256, 0), ("e4m3", 1, 16, 16, 16)]


@pytest.mark.parametrize("kind,h,P,d,T", SHAPES)
def test_copy_pages(kind, h, P, d, T):
    x = pools(20, h, P, d, kind, 1, T)
    moves = [(3, 4, P), (5, 6, 1), (7, 8, 0), (9, 10, P - 1), (0, 19, (P + 1) // 2), (11, 11, P)]
    ref = moved(x, moves, T)
    m = dev(np.array(moves + [(1, 2, P)] * 3))      # the last three are past n_moves
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    nbx.nbx_paged_kv_copy_pages(m, dev([len(moves)]), *x, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(x, ref))


def test_copy_pages_skips_what_is_outside():
    x = pools(8, 2, 16, 64, "bf16", 2)
    ref = moved(x, [(1, 2, 5)])
    for bad, bit in [((8, 3, 4), nbx.DEV_BAD_PAGE), ((3, -1, 4), nbx.DEV_BAD_PAGE), ((3, 4, 17), nbx.DEV_BAD_LEN),
                     ((3, 4, -1), nbx.DEV_BAD_LEN)]:
        y = [t.clone() for t in x]
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        nbx.nbx_paged_kv_copy_pages(dev([bad, (1, 2, 5)]), dev([9]), *y, status=status)   # 9: cut to max_moves
        torch.cuda.synchronize()
        assert int(status.item()) == bit
        assert all(torch.equal(a, b) for a, b in zip(y, ref))


def check_fork(lens, src, dst, P, width, kind="bf16", h=2, d=64, T=0, spread=None, reserve=0, seed=3, bits=0):
    """`spread`: pages of the pool per page in use, and one; by default room for every fork's page."""
    table, n = table_for(lens, P, width, seed, spread=spread or 1.5, reserve=reserve)
    num_pages = n + len(src) if spread is None else n
    x = pools(num_pages, h, P, d, kind, seed, T)
    want_t, want_n, want_m = oc.fork(table, np.array(lens), src, dst, P, num_pages)
    ref = moved(x, want_m, T)
    t, ln = dev(table), dev(lens)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moves, count = nbx.nbx_paged_kv_fork(t, ln, dev(src), dev(dst), *x, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == bits
    assert np.array_equal(t.cpu().numpy(), want_t)
    assert np.array_equal(ln.cpu().numpy(), want_n)
    assert int(count.item()) == len(want_m)
    m = moves.cpu().numpy()
    assert [tuple(r) for r in m[: len(want_m)]] == want_m and np.all(m[len(want_m):] == -1)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(x, ref))
    return t, ln, x


@pytest.mark.parametrize("kind,h,P,d,T", SHAPES)
def test_fork_into_empty_rows(kind, h, P, d, T):
    # lengths of nothing, one position, a full page, a page and one, and longer
    lens = [0, 1, P, P + 1, 5 * P - 1, 3 * P] + [0] * 9
    check_fork(lens, [0, 1, 1, 2, 3, 4, 4, 4, 5], list(range(6, 15)), P, 6, kind, h, d, T)


def test_fork_over_rows_that_hold_pages_frees_them():
    # the destinations' pages are the only free ones
    P = 16
    check_fork([20, 33, 40, 50], [0, 1], [2, 3], P, 4, spread=1.0, seed=5)


def test_beam_reorder_rows_are_read_and_written():
    # every row is a destination: swaps, a row read by several, a row read by none, a row forked to itself
    lens = [20, 33, 47, 50, 64, 5, 17]
    check_fork(lens, [1, 0, 2, 2, 2, 6, 6], [0, 1, 2, 3, 4, 5, 6], 16, 5, seed=6)
    check_fork(lens, [3, 3, 3, 3, 3, 3, 3], [6, 5, 4, 3, 2, 1, 0], 16, 5, seed=7)


def test_reserved_pages_stay_with_their_row_and_are_not_shared():
    check_fork([20, 40, 0, 0], [0, 1], [2, 3], 16, 6, reserve=2, seed=8)


def test_fork_without_free_pages():
    # one page more than is in use: the second copy finds none
    check_fork([20, 33, 0, 0, 0, 0], [0, 1, 0, 1], [2, 3, 4, 5], 16, 3, spread=1.0, seed=9, bits=nbx.DEV_NO_PAGE)


def test_fork_refusals_on_the_device():
    check_fork([20, 33, 7, 0], [0, 4, 1, -1], [3, 2, 9, 2], 16, 3, seed=10, bits=nbx.DEV_BAD_ROW)
    check_fork([20, 33, 0, 0], [0, 1, 1], [2, 2, 3], 16, 3, seed=11, bits=nbx.DEV_BAD_ROW)   # a destination twice


def test_fork_source_length_out_of_bounds():
    table, n = table_for([20, 33, 10, 0], 16, 3, 12)
    lens = np.array([20, 49, -1, 0])            # 49 > 3 pages of 16
    want_t, want_n, want_m = oc.fork(table, lens, [1, 2], [3, 0], 16, n)
    x = pools(n, 1, 16, 64, "bf16", 12)
    t, ln = dev(table), dev(lens)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    nbx.nbx_paged_kv_fork(t, ln, dev([1, 2]), dev([3, 0]), *x, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == nbx.DEV_BAD_LEN
    assert np.array_equal(t.cpu().numpy(), want_t) and np.array_equal(ln.cpu().numpy(), want_n)


def test_many_forks_of_many_rows():
    # more forks and rows than one pass of any step's threads; random trees of forks, with overwritten rows
    g = np.random.default_rng(13)
    B, P, width = 3000, 16, 5
    lens = g.integers(0, width * P + 1, B)
    dst = g.permutation(B)[:1500]
    src = g.integers(0, B, 1500)
    check_fork(list(lens), list(src), list(dst), P, width, h=1, d=16, seed=13)


@pytest.mark.parametrize("kind,h,P,d,T", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(kind, h, P, d, T, in_place):
    g = np.random.default_rng(14)
    lens = list(g.integers(0, 6 * P, 23)) + [0, 1, P]
    table, n = table_for(lens, P, 7, 15, spread=2.3, reserve=1)
    table[3, :4] = table[5, :4]                 # shared pages
    x = pools(n, h, P, d, kind, 16, T)
    want_t, want_m, live = oc.compact(table, lens, P, n)
    ref = moved(x, want_m, T)
    t = dev(table)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    new, moves, counts = nbx.nbx_paged_kv_compact(t, dev(lens), *x, new_block_table=t if in_place else None,
                                                  status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert counts.tolist() == [len(want_m), live]
    assert np.array_equal(new.cpu().numpy(), want_t)
    m = moves.cpu().numpy()
    assert [tuple(r) for r in m[: len(want_m)]] == want_m and np.all(m[len(want_m):] == -1)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(x, ref))


@pytest.mark.parametrize("num_pages", [1, 2, 2047, 2048, 2049, 10000, 24576, 24577, 30000, 70000])
def test_compact_over_the_scan_chunks(num_pages):
    g = np.random.default_rng(num_pages)
    for share in (0.0, 0.5, 1.0):
        used = g.permutation(num_pages)[: int(num_pages * share)].astype(np.int32)
        table = np.full((3, max(1, -(-len(used) // 3))), -1, dtype=np.int32)
        table.reshape(-1)[: len(used)] = used
        lens = [table.shape[1] * 16] * 3
        x = pools(num_pages, 1, 16, 16, "e4m3", 17)
        want_t, want_m, live = oc.compact(table, lens, 16, num_pages)
        ref = moved(x, want_m)
        new, moves, counts = nbx.nbx_paged_kv_compact(dev(table), dev(lens), *x)
        torch.cuda.synchronize()
        assert counts.tolist() == [len(want_m), live]
        assert np.array_equal(new.cpu().numpy(), want_t)
        assert all(torch.equal(a, b) for a, b in zip(x, ref))


def test_compact_a_long_table_of_a_small_pool():
    # more entries than the one-CTA form takes, most of them empty
    g = np.random.default_rng(22)
    table = np.full((900, 80), -1, dtype=np.int32)
    lens = g.integers(0, 80 * 16, 900)
    for i, p in enumerate(g.permutation(3000)[:1500]):
        table[i % 900, i // 900] = p
    x = pools(3000, 1, 16, 16, "bf16", 23)
    want_t, want_m, live = oc.compact(table, lens, 16, 3000)
    ref = moved(x, want_m)
    new, moves, counts = nbx.nbx_paged_kv_compact(dev(table), dev(lens), *x)
    torch.cuda.synchronize()
    assert counts.tolist() == [len(want_m), live] and np.array_equal(new.cpu().numpy(), want_t)
    assert all(torch.equal(a, b) for a, b in zip(x, ref))


def test_fork_then_decode_reads_the_new_lengths():
    # the decode's plan starts while the fork may still run: it has to see the lengths the fork writes, with
    # copies behind them and without (a table-only fork), on both forms of the bookkeeping
    for B in (8, 1200):
        P, d = 16, 64
        lens = [33] * (B // 2) + [0] * (B // 2)
        table, n = table_for(lens, P, 60, 24, spread=2.0)
        k, v = pools(n, 1, P, d, "bf16", 24)
        q = torch.randn((B, 1, 2, d), device=DEV).to(torch.bfloat16)
        q[B // 2:] = q[: B // 2]
        src, dst = dev(np.arange(B // 2)), dev(np.arange(B // 2) + B // 2)
        ws = torch.empty(nbx.nbx_paged_kv_fork_workspace_bytes(B, 60, B // 2, n), dtype=torch.uint8, device=DEV)
        need = nbx.nbx_paged_decode_workspace_bytes(B, 1, 2, 1, d, 64)
        dws = torch.empty(need, dtype=torch.uint8, device=DEV)
        moves = torch.empty((B // 2, 3), dtype=torch.int32, device=DEV)
        count = torch.empty(1, dtype=torch.int32, device=DEV)
        for _ in range(5):
            t, ln = dev(table), dev(lens)
            torch.cuda.synchronize()
            nbx.nbx_paged_kv_fork(t, ln, src, dst, k, v, moves=moves, n_moves=count, workspace=ws)
            out = nbx.nbx_paged_decode_attn(q, k, v, t, ln, 64, 0.125, workspace=dws)
            torch.cuda.synchronize()
            assert torch.equal(out[: B // 2], out[B // 2:])
            t, ln = dev(table), dev(lens)
            args = [t.data_ptr(), 60, ln.data_ptr(), B, src.data_ptr(), dst.data_ptr(), B // 2, None, None, 1, n, 1, P, d,
                    None, None, 0, moves.data_ptr(), count.data_ptr(), ws.data_ptr(), ws.numel(), None]
            torch.cuda.synchronize()
            assert nbx.lib().nbx_paged_kv_fork(*args, torch.cuda.current_stream().cuda_stream) == 0
            shared = nbx.nbx_paged_decode_attn(q, k, v, t, ln, 32, 0.125, workspace=dws)   # full pages alone: len > 32 is
            torch.cuda.synchronize()                                                       # out of bounds, read as empty
            assert ln.tolist() == [33] * B and bool((shared == 0).all())


def test_compact_keeps_entries_outside_the_pool():
    table = np.array([[7, 9, -5, 3]], dtype=np.int32)
    x = pools(8, 1, 16, 16, "f32", 18)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    new, moves, counts = nbx.nbx_paged_kv_compact(dev(table), dev([64]), *x, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == nbx.DEV_BAD_PAGE
    assert new.tolist() == [[1, 9, -5, 0]] and counts.tolist() == [2, 2]


def test_fork_and_compact_captured_and_replayed():
    # one graph: fork, then compact in place; replayed on other contents of the same buffers
    P, width, h, d = 16, 5, 2, 64
    lens = [20, 33, 47, 0, 0, 0]
    src, dst = [0, 1, 1], [3, 4, 5]
    table, n = table_for(lens, P, width, 19, spread=3.0)
    x = pools(n, h, P, d, "bf16", 19)
    t, ln, s, e = dev(table), dev(lens), dev(src), dev(dst)
    moves = torch.full((3, 3), -1, dtype=torch.int32, device=DEV)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)
    m2 = torch.full((n // 2, 3), -1, dtype=torch.int32, device=DEV)
    c2 = torch.zeros(2, dtype=torch.int32, device=DEV)
    w1 = torch.empty(nbx.nbx_paged_kv_fork_workspace_bytes(6, width, 3, n), dtype=torch.uint8, device=DEV)
    w2 = torch.empty(nbx.nbx_paged_kv_compact_workspace_bytes(n), dtype=torch.uint8, device=DEV)

    def step():
        nbx.nbx_paged_kv_fork(t, ln, s, e, *x, moves=moves, n_moves=count, workspace=w1)
        nbx.nbx_paged_kv_compact(t, ln, *x, new_block_table=t, moves=m2, counts=c2, workspace=w2)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (20, 21):
        table, _ = table_for(lens, P, width, seed, spread=3.0)
        y = pools(n, h, P, d, "bf16", seed)
        t.copy_(dev(table))
        ln.copy_(dev(lens))
        for a, b in zip(x, y):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        t1, l1, mv1 = oc.fork(table, np.array(lens), src, dst, P, n)
        ref = moved(y, mv1)
        t2, mv2, live = oc.compact(t1, l1, P, n)
        ref = moved(ref, mv2)
        assert np.array_equal(t.cpu().numpy(), t2) and np.array_equal(ln.cpu().numpy(), l1)
        assert c2.tolist() == [len(mv2), live]
        # what the rows hold, position by position (dropped pages may keep old bits)
        for b in range(6):
            for j in range(int(l1[b])):
                pg = int(t2[b, j // P])
                assert all(torch.equal(a[pg, :, j % P], r[pg, :, j % P]) for a, r in zip(x, ref))


def test_calls_on_another_stream_own_what_they_allocate():
    """Moves and counts that a call allocates for a stream that is not the current one, which is busy."""
    P, width = 16, 5
    lens, src, dst = [20, 33, 47, 0, 0, 0], [0, 1, 1], [3, 4, 5]
    table, n = table_for(lens, P, width, 19, spread=3.0)
    x = pools(n, 2, P, 64, "bf16", 19)
    t, ln, s, e = dev(table), dev(lens), dev(src), dev(dst)
    t1, l1, mv1 = oc.fork(table, np.array(lens), src, dst, P, n)
    t2, mv2, live = oc.compact(t1, l1, P, n)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)   # ten milliseconds or so of the current stream
    m1, c1 = nbx.nbx_paged_kv_fork(t, ln, s, e, *x, stream=side)
    new, m2, c2 = nbx.nbx_paged_kv_compact(t, ln, *x, stream=side)
    torch.cuda.synchronize()
    assert c1.tolist() == [len(mv1)] and [tuple(m) for m in m1[:len(mv1)].tolist()] == mv1
    assert c2.tolist() == [len(mv2), live] and [tuple(m) for m in m2[:len(mv2)].tolist()] == mv2
    assert np.array_equal(t.cpu().numpy(), t1) and np.array_equal(new.cpu().numpy(), t2)


def test_calls_without_rows_or_forks_return_no_moves():
    x = pools(8, 1, 16, 16, "f32", 18)
    none = dev(np.zeros(0))
    m, c = nbx.nbx_paged_kv_fork(dev([[1, 2]]), dev([20]), none, none, *x)
    assert c.tolist() == [0] and m.shape == (0, 3)
    m, c = nbx.nbx_paged_kv_fork(dev(np.zeros((0, 2))), none, dev([0]), dev([1]), *x)
    assert c.tolist() == [0] and m.tolist() == [[-1, -1, -1]]
    new, m, c = nbx.nbx_paged_kv_compact(dev(np.zeros((0, 2))), none, *x)
    assert c.tolist() == [0, 0] and m.tolist() == [[-1, -1, -1]] * 4 and new.shape == (0, 2)


def test_awkward_forks_in_a_table_of_many_rows():
    # the cases above among 300 empty rows, more than one CTA's rows
    rest = [0] * 300
    check_fork([20, 33, 40, 50] + rest, [0, 1], [2, 3], 16, 4, spread=1.0, seed=5)
    lens = [20, 33, 47, 50, 64, 5, 17] + rest
    check_fork(lens, [1, 0, 2, 2, 2, 6, 6], [0, 1, 2, 3, 4, 5, 6], 16, 5, seed=6)
    check_fork(lens, [3, 3, 3, 3, 3, 3, 3], [6, 5, 4, 3, 2, 1, 0], 16, 5, seed=7)
    check_fork([20, 40, 0, 0] + rest, [0, 1], [2, 3], 16, 6, reserve=2, seed=8)
    check_fork([20, 33, 0, 0, 0, 0] + rest, [0, 1, 0, 1], [2, 3, 4, 5], 16, 3, spread=1.0, seed=9, bits=nbx.DEV_NO_PAGE)
    check_fork([20, 33, 7, 0] + rest, [0, 304, 1, -1], [3, 2, 999, 2], 16, 3, seed=10, bits=nbx.DEV_BAD_ROW)
    check_fork([20, 33, 0, 0] + rest, [0, 1, 1], [2, 2, 3], 16, 3, seed=11, bits=nbx.DEV_BAD_ROW)


@pytest.mark.parametrize("rows,width", [(256, 256), (257, 256), (256, 257), (200, 5), (1, 4000)])
def test_fork_around_one_ctas_table(rows, width):
    g = np.random.default_rng(rows + width)
    lens = list(g.integers(0, min(width, 40) * 16 + 1, rows))
    dst = g.permutation(rows)[: max(1, rows // 2)]
    check_fork(lens, list(g.integers(0, rows, len(dst))), list(dst), 16, width, h=1, d=16, seed=rows)


@pytest.mark.parametrize("num_pages", [12287, 12288, 12289])
def test_compact_around_one_ctas_pages(num_pages):
    test_compact_over_the_scan_chunks(num_pages)
