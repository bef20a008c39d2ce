"""kvq_paged_decode_attention_fp4 against the float64 oracle on the cache's
own codes."""
import numpy as np
import pytest
import torch

from tests.fp4_testlib import P, Pool4, assert_within, i32

pytestmark = pytest.mark.gpu


def _k():
    import fp8_kv_cache_reshape_gb300 as k
    return k


def _case(lengths, heads, group, dim, seed=1, window=-1, paired=False, width=None, scale=None, q_factor=1.0):
    pool = Pool4(sum(-(-n // P) for n in lengths) + 3, heads, dim, seed)
    table = pool.table(lengths, width)
    qd, q = pool.query(len(lengths), group)
    if q_factor != 1.0:
        qd = (qd.float() * q_factor).bfloat16()
        q = qd.double().cpu().numpy()
    sm = scale or 1 / np.sqrt(dim)
    args = (qd, *pool.device(paired), *pool.scales(), i32(table), i32(lengths))
    ref, tol = pool.attend(q, table, lengths, sm, window)
    return args, ref, tol, dict(sm_scale=sm, window=window)


def _run(args, kw, **more):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(args[0], 7.0)
    _k().kvq_paged_decode_attention_fp4(*args, out, dev_status=st, **kw, **more)
    torch.cuda.synchronize()
    return out, int(st)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lengths", [[1], [0], [16], [17], [15, 0, 0, 33], [63, 64, 65, 1000], [2500], [0, 0, 5, 0, 700, 0]])
def test_lengths(lengths, dim):
    args, ref, tol, kw = _case(lengths, 2, 4, dim)
    out, st = _run(args, kw)
    assert st == 0
    assert_within(out, ref, tol)
    for b, n in enumerate(lengths):
        if n == 0:
            assert not out[b].any()


@pytest.mark.parametrize("heads,group,dim", [(1, 1, 64), (3, 3, 128), (8, 8, 64), (5, 7, 128), (1, 8, 128)])
def test_heads(heads, group, dim):
    args, ref, tol, kw = _case([130, 1, 577], heads, group, dim, paired=True)
    out, st = _run(args, kw)
    assert st == 0
    assert_within(out, ref, tol)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 129, 5000])
@pytest.mark.parametrize("dim", [64, 128])
def test_window(window, dim):
    args, ref, tol, kw = _case([1, 16, 130, 777, 0], 2, 4, dim, window=window)
    out, st = _run(args, kw)
    assert st == 0
    assert_within(out, ref, tol)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lengths", [[1, 40], [9000, 333]])
def test_a_nan_block_shows_and_stays_where_it_is(lengths, dim):
    """What the write makes of a NaN: its key's scores, and so the head's outputs, and its value's 16 dims."""
    heads, group = 2, 3
    pool = Pool4(sum(-(-n // P) for n in lengths) + 3, heads, dim, 5)
    table = pool.table(lengths)
    qd, q = pool.query(2, group)
    sm = 1 / np.sqrt(dim)
    ref, tol = pool.attend(q, table, lengths, sm)
    last = lengths[0] - 1
    pool.ks[table[0, last // P], 0, last % P, 1] = 0x7F
    pool.vs[table[0, 0], 1, 0, 2] = 0x7F
    args = (qd, *pool.device(), *pool.scales(), i32(table), i32(lengths))
    out, st = _run(args, dict(sm_scale=sm, window=-1))
    assert st == 0
    odd = torch.zeros(out.shape, dtype=torch.bool)
    odd[0, :group] = True
    odd[0, group:, 32:48] = True
    assert torch.equal(out.isnan().cpu(), odd)
    ref[odd.numpy()] = 0
    assert_within(out.nan_to_num(0.0), ref, tol)


def test_more_sequences_than_threads_of_a_cta():
    """Most of them empty, the rest at both ends."""
    lengths = [0] * 300
    lengths[0], lengths[131], lengths[299] = 40, 19, 133
    args, ref, tol, kw = _case(lengths, 2, 2, 64)
    out, st = _run(args, kw)
    assert st == 0
    assert_within(out, ref, tol)


@pytest.mark.parametrize("lengths,dim", [([70, 0, 5], 128), ([1], 64), ([333] * 9, 64)])
def test_a_table_much_wider_than_the_sequences(lengths, dim):
    """Parts without pages, and CTAs without parts."""
    args, ref, tol, kw = _case(lengths, 3, 2, dim, width=1500)
    out, st = _run(args, kw)
    assert st == 0
    assert_within(out, ref, tol)


def test_many_short_sequences():
    lengths = [1 + (37 * b) % 75 for b in range(400)]
    args, ref, tol, kw = _case(lengths, 2, 4, 64)
    out, st = _run(args, kw)
    assert st == 0
    assert_within(out, ref, tol)


@pytest.mark.parametrize("factor", [0.0, 1e-20, 40.0])
def test_query_scales(factor):
    """No scores, scores of nothing, and weights on a few tokens."""
    args, ref, tol, kw = _case([900, 3], 2, 4, 128, q_factor=factor)
    out, st = _run(args, kw)
    assert st == 0
    # scores of up to about 40 * 1.5 * 6 * sqrt(128) * log2 e / sqrt(128), 520 in base 2: their float32 steps, 2^-15 each,
    # on the product and on its difference from the stabilizer, move a weight by 2^-14
    assert_within(out, ref, tol * (1 + 2.0 ** -2) if factor > 1 else tol)


def test_descending_and_ascending_scores():
    """The stabilizer is the first page's, or moves with every page."""
    for sign in (1, -1):
        pool = Pool4(70, 1, 64, 5)
        n = 1000
        table = pool.table([n])
        j = np.arange(n)
        at, off = table[0, j // P], j % P
        x = np.zeros((n, 64), np.float32)
        x[:, 0] = 6 * sign * (j / n - 0.5)
        x[:, 1:] = 0.1 * np.random.default_rng(3).standard_normal((n, 63))
        from oracle import e2m1
        pool.k[at, 0, off], pool.ks[at, 0, off] = e2m1.quantize(x, pool.k_scale[0])
        qd = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
        qd[0, :, 0] = torch.tensor([9.0, -30.0])
        args = (qd, *pool.device(), *pool.scales(), i32(table), i32([n]))
        ref, tol = pool.attend(qd.double().cpu().numpy(), table, [n], 1.0)
        out, st = _run(args, dict(sm_scale=1.0))
        assert st == 0
        assert_within(out, ref, tol)


def test_bad_blocks_are_masked():
    pool = Pool4(20, 2, 128, 7)
    lengths = [100, 40]
    table = pool.table(lengths)
    qd, q = pool.query(2, 4)
    bad = {(0, 0): -1, (0, 3): 20, (0, 6): 2**31 - 1, (1, 0): -5, (1, 1): 99, (1, 2): 21}
    broken = table.copy()
    for (b, j), v in bad.items():
        broken[b, j] = v
    args = (qd, *pool.device(), *pool.scales(), i32(broken), i32(lengths))
    ref, tol = pool.attend(q, table, lengths, 128 ** -0.5, bad=bad)
    out, st = _run(args, {})
    assert st == _k().KVQ_DEV_BAD_BLOCK
    assert_within(out, ref, tol)
    assert not out[1].any()


def test_bad_lengths_are_clamped():
    pool = Pool4(20, 2, 64, 8)
    table = pool.table([64, 64])
    qd, q = pool.query(2, 2)
    args = (qd, *pool.device(), *pool.scales(), i32(table), i32([1000, -3]))
    ref, tol = pool.attend(q, table, [64, 0], 0.125)
    out, st = _run(args, {})
    assert st == _k().KVQ_DEV_BAD_SEQLEN
    assert_within(out, ref, tol)


def test_same_bits_whatever_the_workspace_holds():
    args, ref, tol, kw = _case([3000, 20, 0, 411], 4, 4, 128)
    size = _k().kvq_decode_fp4_workspace_size(4, 16, 4, 128, args[5].shape[1])
    first, _ = _run(args, kw)
    assert_within(first, ref, tol)
    for fill in (0, 0xFF, 0x7F):
        out, st = _run(args, kw, workspace=torch.full((size,), fill, dtype=torch.uint8, device="cuda"))
        assert st == 0 and torch.equal(out, first)


def test_graphs_that_share_a_workspace_and_a_side_stream():
    """Two captured calls replayed in turn, and an eager one on another stream beside them with a workspace of its own."""
    k = _k()
    one, two = _case([1500, 9], 2, 4, 64, seed=2), _case([33, 2000], 2, 4, 64, seed=3)
    size = max(k.kvq_decode_fp4_workspace_size(2, 8, 2, 64, c[0][5].shape[1]) for c in (one, two))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for args, _, _, kw in (one, two):
        out = torch.zeros_like(args[0])
        k.kvq_paged_decode_attention_fp4(*args, out, workspace=ws, **kw)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            k.kvq_paged_decode_attention_fp4(*args, out, workspace=ws, **kw)
        graphs.append(g)
        outs.append(out)
    side = torch.cuda.Stream()
    for _ in range(3):
        eager = torch.zeros_like(outs[0])
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        k.kvq_paged_decode_attention_fp4(*one[0], eager, stream=side, **one[3])
        torch.cuda.synchronize()
        for o, c in zip(outs, (one, two)):
            assert_within(o, c[1], c[2])
        assert torch.equal(eager, outs[0])


def test_memory_given_back_by_another_stream_is_left_alone():
    """A call without a workspace on a side stream, while the current stream still writes memory that it has given back."""
    k = _k()
    args, ref, tol, kw = _case([2000, 31, 700], 2, 4, 128)
    alone, _ = _run(args, kw)
    size = k.kvq_decode_fp4_workspace_size(3, 8, 2, 128, args[5].shape[1])
    side, big, out = torch.cuda.Stream(), torch.ones(4096, 4096, device="cuda"), torch.zeros_like(alone)
    torch.cuda.synchronize()
    given_back = torch.empty(size, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        big @ big
    for _ in range(300):
        given_back.fill_(0xFF)
    del given_back
    k.kvq_paged_decode_attention_fp4(*args, out, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out, alone)


@pytest.mark.parametrize("lengths,heads,group", [([20000], 1, 8), ([30000, 5], 8, 4), ([4096] * 3, 4, 2)])
def test_long(lengths, heads, group):
    """Many pieces to a row, whole CTAs of one sequence and KV head, and parts that end in others."""
    args, ref, tol, kw = _case(lengths, heads, group, 128)
    out, st = _run(args, kw)
    assert st == 0
    assert_within(out, ref, tol)


def test_offsets_beyond_32_bits():
    """A cache of more than 4 GiB per tensor, its last pages used."""
    k = _k()
    blocks, heads = 3_800_000, 1
    kd, vd = k.alloc_kv_cache(blocks, heads, 128, "fp4")
    assert kd.nbytes > 2**32
    pool = Pool4(12, heads, 128, 9)
    table = pool.table([150])
    small = pool.device()
    place = torch.arange(blocks - 12, blocks, device="cuda")
    kd[place], vd[place] = small[0], small[1]
    qd, q = pool.query(1, 4)
    ref, tol = pool.attend(q, table, [150], 128 ** -0.5)
    out, st = _run((qd, kd, vd, *pool.scales(), i32(table + blocks - 12), i32([150])), {})
    assert st == 0
    assert_within(out, ref, tol)
