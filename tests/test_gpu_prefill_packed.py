"""GPU tests of the packed prefills: sequences of different lengths, dense and over the paged cache."""
import numpy as np
import pytest
import torch

from oracle import sdpa
from packed_oracle import assert_packed, cumulative, f64, packed_attention
from scaled_dot_product_prefill_b200 import api, inputs

pytestmark = pytest.mark.gpu


def run_packed(q, k, v, cu_q, cu_k=None, **kw):
    api.attn_device_status(clear=True)
    got = api.attn_prefill_packed(q.cuda(), k.cuda(), v.cuda(), cu_q.cuda(), None if cu_k is None else cu_k.cuda(),
                                  want_lse=True, **kw)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    return got


def tensors(Tq, Tk, Hq, Hkv, D, seed):
    return (inputs.normal((Tq, Hq, D), seed), inputs.normal((Tk, Hkv, D), seed + 1),
            inputs.normal((Tk, Hkv, D), seed + 2))


SELF = [
    # Hq, Hkv, D, lengths, causal, window
    (4, 4, 64, [1], True, 0),
    (8, 2, 128, [1], True, 0),
    (8, 2, 128, [1, 1, 1, 1, 1], True, 0),
    (4, 4, 64, [0, 5, 0, 130, 128, 127, 129, 0], True, 0),
    (8, 2, 128, [0, 5, 0, 130, 128, 127, 129, 0], True, 0),
    (8, 1, 128, [256, 255, 257, 33, 31, 32], True, 0),
    (8, 1, 64, [17, 300, 16, 15], True, 0),
    (12, 4, 128, [100, 260], True, 0),           # groups of 3: no shared tiles
    (6, 1, 64, [90, 1, 200], True, 0),           # groups of 6: pairs of heads share a tile
    (5, 5, 128, [140], True, 0),
    (16, 1, 128, [70, 20], True, 0),
    (32, 1, 64, [40, 5], True, 0),
    (128, 1, 64, [3, 6], True, 0),               # a tile is one token
    (8, 2, 64, [400, 130], True, 1),             # a window of the token itself
    (8, 2, 128, [400, 130], True, 7),
    (4, 1, 128, [700, 10], True, 128),
    (4, 2, 64, [513, 300], True, 200),
    (4, 2, 128, [300, 20], True, 2 ** 31 - 1),   # a window longer than anything
    (8, 2, 128, [200, 0, 77, 1], False, 0),
    (4, 4, 64, [128, 129, 300], False, 0),
]


@pytest.mark.parametrize("case", SELF, ids=[str(c) for c in SELF])
def test_packed_prefill_matches_the_definition(case):
    Hq, Hkv, D, lens, causal, window = case
    T = sum(lens)
    q, k, v = tensors(T, T, Hq, Hkv, D, seed=T + Hq)
    cu = cumulative(lens)
    got = run_packed(q, k, v, cu, causal=causal, window=window)
    assert_packed(got, packed_attention(f64(q), f64(k), f64(v), cu.tolist(), cu.tolist(), D ** -0.5, causal, window),
                  str(case))


CROSS = [
    # Hq, Hkv, D, query lengths, key lengths, causal, window
    (8, 2, 128, [5, 130, 1], [300, 130, 513], True, 0),
    (8, 2, 64, [300, 40, 129], [10, 0, 128], True, 0),        # rows that see nothing, a sequence without keys
    (4, 4, 128, [0, 300, 7], [50, 20, 0], True, 0),           # a sequence without queries
    (4, 1, 128, [60, 200], [1000, 900], True, 130),
    (4, 2, 64, [200, 3], [150, 70], True, 5),
    (4, 2, 128, [33, 150, 9], [200, 0, 129], False, 0),
    (6, 2, 64, [200], [1], True, 0),
]


@pytest.mark.parametrize("case", CROSS, ids=[str(c) for c in CROSS])
def test_queries_and_keys_of_different_lengths(case):
    Hq, Hkv, D, lq, lk, causal, window = case
    q, k, v = tensors(sum(lq), sum(lk), Hq, Hkv, D, seed=7 + sum(lk))
    cu_q, cu_k = cumulative(lq), cumulative(lk)
    got = run_packed(q, k, v, cu_q, cu_k, causal=causal, window=window, scale=0.11)
    assert_packed(got, packed_attention(f64(q), f64(k), f64(v), cu_q.tolist(), cu_k.tolist(), 0.11, causal, window),
                  str(case))


def test_no_keys_at_all():
    q, _, _ = tensors(40, 0, 4, 2, 64, 3)
    kv = torch.empty((0, 2, 64), dtype=torch.bfloat16)
    out, lse = run_packed(q, kv, kv, cumulative([30, 10]), cumulative([0, 0]))
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (128, 150)])
def test_many_sequences_more_items_than_sms(D, window):
    r = np.random.default_rng(4)
    lens = r.integers(0, 300, 70).tolist()
    T = sum(lens)
    q, k, v = tensors(T, T, 8, 4, D, seed=11)
    cu = cumulative(lens)
    got = run_packed(q, k, v, cu, window=window)
    assert_packed(got, packed_attention(f64(q), f64(k), f64(v), cu.tolist(), cu.tolist(), D ** -0.5, True, window))
    # each sequence alone gives the same bits: nothing depends on its neighbours or its place
    for b in (0, 13, 69):
        a, e = int(cu[b]), int(cu[b + 1])
        if a == e:
            continue
        one = api.attn_prefill_packed(q[a:e].cuda(), k[a:e].cuda(), v[a:e].cuda(), cumulative([e - a]).cuda(),
                                      window=window)
        assert torch.equal(one, got[0][a:e])


@pytest.mark.parametrize("causal", [True, False])
def test_thousands_of_sequences_beside_a_long_one(causal):
    """More sequences than one pass of the scheduler's warp holds, and steps of cost folded into levels."""
    r = np.random.default_rng(8)
    lens = r.integers(0, 5, 4000)
    lens[1234], lens[3999] = 2500, 700
    T, Hq, Hkv, D = int(lens.sum()), 4, 1, 64
    q, k, v = (x.cuda() for x in tensors(T, T, Hq, Hkv, D, seed=5))
    cu = cumulative(lens)
    out, lse = api.attn_prefill_packed(q, k, v, cu.cuda(), causal=causal, want_lse=True)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    want = packed_attention(f64(q), f64(k), f64(v), cu.tolist(), cu.tolist(), D ** -0.5, causal)
    assert_packed((out, lse), want)


@pytest.mark.parametrize("D,Hq,Hkv,causal,window", [(64, 4, 4, True, 0), (128, 8, 2, True, 0), (128, 8, 2, True, 300),
                                                    (64, 4, 1, False, 0)])
def test_equal_lengths_give_the_bits_of_the_dense_prefill(D, Hq, Hkv, causal, window):
    B, S = 3, 777
    p = inputs.prefill_inputs(B, Hq, Hkv, S, S, D, seed=8)
    dense, dense_lse = api.attn_prefill_lse(p.q.cuda(), p.k.cuda(), p.v.cuda(), causal=causal, window=window)
    rows = lambda x: x.transpose(1, 2).reshape(B * S, x.shape[1], D).contiguous()  # noqa: E731
    out, lse = run_packed(rows(p.q), rows(p.k), rows(p.v), cumulative([S] * B), causal=causal, window=window)
    assert torch.equal(out.view(B, S, Hq, D).transpose(1, 2), dense)
    assert torch.equal(lse.view(B, S, Hq).transpose(1, 2), dense_lse)


@pytest.mark.parametrize("D", [64, 128])
def test_what_lies_around_a_sequence_never_reaches_it(D):
    """NaN before the first sequence, in the middle one and behind the last: the others keep their bits, the rows of no
    sequence keep what they held."""
    Hq, Hkv, lens, front, back = 8, 2, [75, 140, 130, 1, 60], 9, 200
    T = front + sum(lens) + back
    q, k, v = tensors(T, T, Hq, Hkv, D, seed=21)
    cu = cumulative(lens, front)
    clean = run_packed(q, k, v, cu)
    mine = torch.zeros(T, dtype=torch.bool)
    for b in (0, 2, 3, 4):
        mine[int(cu[b]):int(cu[b + 1])] = True
    for x in (q, k, v):
        x[~mine] = float("nan")
        x[int(cu[1]):int(cu[2])][::3] = float("inf")
    out = torch.full((T, Hq, D), 3.5, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), -7.25, device="cuda")
    run_packed(q, k, v, cu, out=out, lse=lse)
    assert torch.equal(out[mine.cuda()], clean[0][mine.cuda()])
    assert torch.equal(lse[mine.cuda()], clean[1][mine.cuda()])
    for edge in (slice(0, front), slice(T - back, T)):
        assert (out[edge] == 3.5).all() and (lse[edge] == -7.25).all()


def test_masked_keys_with_nan_scores_are_never_seen():
    """NaN and infinities in K rows that a query does not see stay out of it (V finite there)."""
    q, k, v = tensors(300, 300, 4, 2, 128, 31)
    cu = cumulative([300])
    clean = run_packed(q, k, v, cu)
    k[200:] = float("nan")
    k[250:] = float("inf")
    out, lse = run_packed(q, k, v, cu)
    assert torch.equal(out[:200], clean[0][:200]) and torch.equal(lse[:200], clean[1][:200])


def test_slices_of_a_fused_projection_and_a_strided_output():
    Hq, Hkv, D, lens = 8, 2, 128, [33, 190, 64]
    T = sum(lens)
    qkv = inputs.normal((T, (Hq + 2 * Hkv) * D + 40), 5).cuda()
    cut = lambda a, h: qkv[:, a:a + h * D].view(T, h, D)  # noqa: E731
    q, k, v = cut(0, Hq), cut(Hq * D, Hkv), cut((Hq + Hkv) * D, Hkv)
    wide = torch.full((T, Hq * D + 24), 2.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 8:8 + Hq * D].view(T, Hq, D)
    cu = cumulative(lens).cuda()
    api.attn_prefill_packed(q, k, v, cu, out=out)
    want = api.attn_prefill_packed(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert (wide[:, :8] == 2).all() and (wide[:, 8 + Hq * D:] == 2).all()


def test_scores_far_apart_and_large():
    """Scores of thousands: the reference maximum moves by far more than the exponent's range."""
    Hq, Hkv, D, lens = 4, 2, 64, [150, 300]
    T = sum(lens)
    q, k, v = tensors(T, T, Hq, Hkv, D, 41)
    q, k = q * 32, k * 32
    cu = cumulative(lens)
    got = run_packed(q, k, v, cu)
    assert_packed(got, packed_attention(f64(q), f64(k), f64(v), cu.tolist(), cu.tolist(), D ** -0.5))


PAGED = [
    # Hq, Hkv, D, page, new tokens, cached tokens (new ones included), causal, window
    (8, 2, 128, 16, [77, 1, 0, 300], [77, 300, 40, 1000], True, 0),
    (4, 4, 64, 32, [256, 5, 1], [256, 700, 1], True, 0),
    (8, 1, 128, 64, [130, 20], [40, 513], True, 0),            # a cache shorter than the chunk
    (8, 2, 64, 128, [300, 64], [1500, 300], True, 200),
    (4, 2, 128, 256, [200, 33], [600, 201], False, 0),
    (4, 2, 64, 256, [100, 9], [129, 250], True, 0),            # 127 and 6 NaN slots in the last 128-row box
    (6, 2, 128, 16, [30, 3], [0, 140], True, 0),               # an empty cache
    (12, 4, 64, 16, [1, 1, 1, 1], [1, 128, 129, 515], True, 0),
    (16, 1, 128, 32, [40], [127], True, 33),
]


def gathered(p, lens):
    """The caches of all sequences, packed one after another, in float64."""
    ks, vs = [], []
    for b, L in enumerate(lens):
        for pool, to in ((p.k_pool, ks), (p.v_pool, vs)):
            to.append(sdpa.gather_pages(pool, p.page_table[b].numpy(), L, p.page_size))
    return np.concatenate(ks), np.concatenate(vs)


@pytest.mark.parametrize("case", PAGED, ids=[str(c) for c in PAGED])
def test_packed_chunks_over_the_paged_cache(case):
    Hq, Hkv, D, page, new, lens, causal, window = case
    p = inputs.paged_inputs(len(lens), Hq, Hkv, D, page, seed=sum(lens) + D, seq_lens=lens, spare_pages=3, poison=True)
    q = inputs.normal((sum(new) + 5, Hq, D), 77)
    q[sum(new):] = float("nan")
    cu = cumulative(new)
    api.attn_device_status(clear=True)
    got = api.attn_prefill_packed_paged(q.cuda(), p.k_pool.cuda(), p.v_pool.cuda(), cu.cuda(), p.page_table.cuda(),
                                        p.seq_lens.cuda(), max_seq_len=max(lens), causal=causal, window=window,
                                        want_lse=True)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    K, V = gathered(p, lens)
    assert_packed(got, packed_attention(f64(q), K, V, cu.tolist(), cumulative(lens).tolist(), D ** -0.5, causal,
                                        window), str(case))


def test_paged_and_dense_packed_agree_to_the_bit():
    Hq, Hkv, D, page, lens = 8, 2, 128, 16, [300, 17, 129]
    p = inputs.paged_inputs(3, Hq, Hkv, D, page, seed=3, seq_lens=lens)
    q = inputs.normal((sum(lens), Hq, D), 5).cuda()
    K, V = (torch.from_numpy(x).to(torch.bfloat16).cuda() for x in gathered(p, lens))
    cu = cumulative(lens).cuda()
    dense = api.attn_prefill_packed(q, K, V, cu, window=100)
    paged = api.attn_prefill_packed_paged(q, p.k_pool.cuda(), p.v_pool.cuda(), cu, p.page_table.cuda(),
                                          p.seq_lens.cuda(), max_seq_len=300, window=100)
    torch.cuda.synchronize()
    assert torch.equal(dense, paged)


def test_an_empty_cache_of_no_pages():
    q = inputs.normal((9, 4, 64), 1).cuda()
    pool = torch.empty((0, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = api.attn_prefill_packed_paged(q, pool, pool, cumulative([4, 5]).cuda(),
                                             torch.empty((2, 0), dtype=torch.int32, device="cuda"),
                                             torch.zeros(2, dtype=torch.int32, device="cuda"), max_seq_len=0,
                                             want_lse=True)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_a_bad_page_is_reported_and_not_read():
    lens, new = [100, 60], [30, 20]
    p = inputs.paged_inputs(2, 4, 2, 64, 16, seed=2, seq_lens=lens)
    table = p.page_table.clone()
    table[0, 3] = p.num_pages + 77
    table[0, 5] = -4
    q = inputs.normal((50, 4, 64), 3)
    cu = cumulative(new)
    api.attn_device_status(clear=True)
    out, lse = api.attn_prefill_packed_paged(q.cuda(), p.k_pool.cuda(), p.v_pool.cuda(), cu.cuda(), table.cuda(),
                                             p.seq_lens.cuda(), max_seq_len=100, want_lse=True)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 5
    K, V = gathered(p, lens)
    want = packed_attention(f64(q), K, V, cu.tolist(), cumulative(lens).tolist(), 1 / 8)
    ok = [w[30:] for w in want]
    assert_packed((out[30:], lse[30:]), ok, "the other sequence")


@pytest.mark.parametrize("cu", [[0, 60, 40, 100], [0, 30, 60, 400], [-20, 10, 60, 100], [0, 2 ** 31 - 1, 5, -2 ** 31]])
def test_malformed_cumulative_lengths_are_reported_and_stay_in_the_buffers(cu):
    q, k, v = (x.cuda() for x in tensors(100, 100, 4, 2, 64, 3))
    guard = torch.full((300, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    out = guard[100:200]
    api.attn_device_status(clear=True)
    api.attn_prefill_packed(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 5
    assert (guard[:100] == 9).all() and (guard[200:] == 9).all()
    # the library goes on as before
    good = cumulative([40, 60])
    got = run_packed(q.cpu(), k.cpu(), v.cpu(), good)
    assert_packed(got, packed_attention(f64(q), f64(k), f64(v), good.tolist(), good.tolist(), 1 / 8))


def test_a_sequence_longer_than_max_seq_len_is_cut_and_reported():
    p = inputs.paged_inputs(1, 4, 2, 64, 16, seed=2, seq_lens=[100])
    q = inputs.normal((10, 4, 64), 3).cuda()
    api.attn_device_status(clear=True)
    out = api.attn_prefill_packed_paged(q, p.k_pool.cuda(), p.v_pool.cuda(), cumulative([10]).cuda(),
                                        p.page_table.cuda(), p.seq_lens.cuda(), max_seq_len=64)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 5
    assert torch.isfinite(out.float()).all()


def test_a_captured_graph_is_replayed_with_other_lengths_while_another_runs():
    Hq, Hkv, D, T = 8, 2, 128, 600
    q, k, v = (x.cuda() for x in tensors(T, T, Hq, Hkv, D, 50))
    streams, graphs, cus, outs = [], [], [], []
    for i in range(2):
        cu = cumulative([100, 100, 100, 100, 100]).cuda()
        out = torch.zeros_like(q)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            api.attn_prefill_packed(q, k, v, cu, out=out)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.attn_prefill_packed(q, k, v, cu, out=out)
        streams.append(s), graphs.append(g), cus.append(cu), outs.append(out)
    for lens in ([600, 0, 0, 0, 0], [1, 2, 3, 4, 5], [0, 0, 0, 0, 0], [120, 120, 120, 120, 120]):
        other = [x // 2 for x in lens]
        for cu, n, out in zip(cus, (lens, other), outs):
            cu.copy_(cumulative(n))
            out.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):       # both in flight at once
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert api.attn_device_status(clear=True) == 0
        for n, out in ((lens, outs[0]), (other, outs[1])):
            eager = torch.zeros_like(q)
            api.attn_prefill_packed(q, k, v, cumulative(n).cuda(), out=eager)
            torch.cuda.synchronize()
            assert torch.equal(eager, out)
    del graphs


def test_arguments_beyond_a_c_int_mean_what_they_say_or_are_refused():
    q, k, v = (x.cuda() for x in tensors(200, 200, 4, 2, 64, 60))
    cu = cumulative([150, 50]).cuda()
    want = api.attn_prefill_packed(q, k, v, cu)
    assert torch.equal(api.attn_prefill_packed(q, k, v, cu, window=2 ** 32 + 5), want)
    pool, table, lens = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda"), \
        torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw, status in ((dict(max_seq_len=2 ** 32 + 16), 2), (dict(max_seq_len=-2 ** 40), 1),
                       (dict(max_seq_len=16, window=-2 ** 40), 1), (dict(max_seq_len=16, scale=1e300), 1),
                       (dict(max_seq_len=16, scale=float("nan")), 1)):
        with pytest.raises(api.AttnError) as e:
            api.attn_prefill_packed_paged(q, pool, pool, cu, table, lens, **kw)
        assert e.value.status == status


def test_a_call_on_another_stream_with_its_own_result():
    q, k, v = (x.cuda() for x in tensors(500, 500, 8, 2, 64, 60))
    cu = cumulative([300, 200]).cuda()
    want = api.attn_prefill_packed(q, k, v, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = api.attn_prefill_packed(q, k, v, cu, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


SPLIT = [
    # Hq, Hkv, D, page (0: packed keys), query lengths, key lengths, causal, window
    (8, 2, 128, 16, [5, 1], [3000, 1100], True, 0),
    (8, 2, 64, 0, [9, 3, 0], [2500, 4, 700], True, 0),          # parts without keys; a sequence without queries
    (4, 1, 128, 0, [40, 200], [2048, 30], True, 0),             # rows that see nothing
    (16, 16, 64, 32, [1], [4097], True, 0),
    (8, 1, 128, 64, [33, 2], [2000, 1500], True, 600),          # most parts lie before the window
    (4, 4, 128, 256, [3, 17], [1500, 2600], False, 0),
    (6, 2, 64, 128, [20], [1025], True, 0),
    (2, 1, 128, 0, [130, 1], [5000, 0], True, 0),
]


@pytest.mark.parametrize("case", SPLIT, ids=[str(c) for c in SPLIT])
def test_few_rows_over_long_sequences_are_split_and_joined(case):
    Hq, Hkv, D, page, lq, lk, causal, window = case
    Tq, cu_q, cu_k = sum(lq) + 3, cumulative(lq, 1), cumulative(lk)
    q = inputs.normal((Tq, Hq, D), 5)
    out = torch.full((Tq, Hq, D), 3.5, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Tq, Hq), -7.25, device="cuda")
    bound = max(lk) if page else -(-sum(lk) // len(lk))
    need = api.attn_prefill_packed_workspace_size(len(lq), Tq, Hq, Hkv, D, bound)
    assert need > 0
    # a workspace that has been used before: full of NaN
    ws = torch.full((need // 4,), float("nan"), device="cuda").view(torch.uint8)
    api.attn_device_status(clear=True)
    if page:
        p = inputs.paged_inputs(len(lk), Hq, Hkv, D, page, seed=9, seq_lens=lk, spare_pages=3, poison=True)
        K, V = gathered(p, lk)
        call = lambda **kw: api.attn_prefill_packed_paged(  # noqa: E731
            q.cuda(), p.k_pool.cuda(), p.v_pool.cuda(), cu_q.cuda(), p.page_table.cuda(), p.seq_lens.cuda(),
            max_seq_len=max(lk), causal=causal, window=window, **kw)
    else:
        k, v = inputs.normal((sum(lk), Hkv, D), 6), inputs.normal((sum(lk), Hkv, D), 7)
        K, V = f64(k), f64(v)
        call = lambda **kw: api.attn_prefill_packed(  # noqa: E731
            q.cuda(), k.cuda(), v.cuda(), cu_q.cuda(), cu_k.cuda(), causal=causal, window=window, **kw)
    call(out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    assert_packed((out, lse), packed_attention(f64(q), K, V, cu_q.tolist(), cu_k.tolist(), D ** -0.5, causal, window),
                  str(case))
    for edge in (slice(0, 1), slice(Tq - 2, Tq)):
        assert (out[edge] == 3.5).all() and (lse[edge] == -7.25).all()
    # the same bits from a workspace made in the call
    again, again_lse = call(want_lse=True)
    held = slice(1, Tq - 2)
    assert torch.equal(again[held], out[held]) and torch.equal(again_lse[held], lse[held])


def test_a_split_row_whose_scores_are_nan_is_nan():
    q, k, v = tensors(2, 3000, 4, 1, 128, 3)
    k[40] = float("nan")
    out, lse = api.attn_prefill_packed(q.cuda(), k.cuda(), v.cuda(), cumulative([2]).cuda(), cumulative([3000]).cuda(),
                                       want_lse=True)
    torch.cuda.synchronize()
    assert torch.isnan(out.float()).all() and torch.isnan(lse).all()


def test_without_a_workspace_nothing_is_split():
    """The C call with a NULL workspace gives the rows to one SM each; the result is as good."""
    import ctypes

    from scaled_dot_product_prefill_b200 import _lib

    Hq, Hkv, D, lk = 8, 2, 128, [3000]
    q, k, v = (x.cuda() for x in tensors(4, 3000, Hq, Hkv, D, 3))
    cu_q, cu_k = cumulative([4]).cuda(), cumulative(lk).cuda()
    out, lse = torch.empty_like(q), torch.empty((4, Hq), device="cuda")
    st = _lib.load().attn_prefill_packed(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(), 1, 4, 3000, Hq, Hkv, D, Hq * D,
        Hkv * D, Hkv * D, Hq * D, D ** -0.5, 1, 0, None, 0, out.data_ptr(), lse.data_ptr(),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and api.attn_device_status(clear=True) == 0
    assert_packed((out, lse), packed_attention(f64(q), f64(k), f64(v), [0, 4], [0, 3000], D ** -0.5))


def test_split_calls_in_two_replayed_graphs_do_not_share_their_workspaces():
    Hq, Hkv, D = 8, 2, 128
    q, k, v = (x.cuda() for x in tensors(8, 4000, Hq, Hkv, D, 3))
    cu_k = cumulative([4000]).cuda()
    graphs, outs, streams = [], [], []
    for i in range(2):
        cu = cumulative([8 - 3 * i]).cuda()
        ws = torch.empty(api.attn_prefill_packed_workspace_size(1, 8, Hq, Hkv, D, 4000), dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(q)
        fn = lambda: api.attn_prefill_packed(q, k, v, cu, cu_k, out=out, workspace=ws)  # noqa: E731, B023
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            fn()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        graphs.append((g, cu, ws)), outs.append((out, out.clone())), streams.append(s)
    torch.cuda.synchronize()
    want = [o.clone() for o, _ in outs]
    for _ in range(5):
        for o, _ in outs:
            o.zero_()
        torch.cuda.synchronize()
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for (o, _), w in zip(outs, want))
    assert api.attn_device_status(clear=True) == 0
    del graphs


@pytest.mark.parametrize("D", [64, 128])
def test_a_call_on_another_stream_is_not_overwritten_by_work_queued_on_this_one(D):
    """The current stream still has to fill blocks that were released on the host: no result or workspace made
    by a call on another stream may lie in them."""
    Hq, Hkv, n, L = 8, 2, 16, 3000
    q, k, v = (x.cuda() for x in tensors(n, L, Hq, Hkv, D, 3))
    cu_q, cu_k = cumulative([n]).cuda(), cumulative([L]).cuda()
    want = api.attn_prefill_packed(q, k, v, cu_q, cu_k, want_lse=True)
    p = inputs.paged_inputs(1, Hq, Hkv, D, 16, seed=3, seq_lens=[L])
    kp, vp, pt, sl = (x.cuda() for x in (p.k_pool, p.v_pool, p.page_table, p.seq_lens))
    kn, vn = k[:n].clone(), v[:n].clone()
    turned = api.attn_kv_append_rope(q, kn, vn, kp, vp, None, pt, sl)
    s = torch.cuda.Stream()
    need = api.attn_prefill_packed_workspace_size(1, n, Hq, Hkv, D, L)
    assert need > 0
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)             # some 50 ms
    for _ in range(2):
        for size in (q.numel() * 2, n * Hq * 4, need):
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
    out, lse = api.attn_prefill_packed(q, k, v, cu_q, cu_k, want_lse=True, stream=s)
    again = api.attn_kv_append_rope(q, kn, vn, kp, vp, None, pt, sl, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(again, turned)
    assert api.attn_device_status(clear=True) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_an_item_may_last_longer_than_any_wait_is_allowed_to(D):
    """One row over 2^28 keys on one SM, some 3 s: the roles that wait for the end of the item go on waiting as long as
    key tiles pass (a wait without progress ends after 2 s).

    The page table names page 0 over and over, with scores of 0 and v that alternates in sign, and page 1
    at the end, whose 156 keys weigh e^28 or more each: the result is the mean of their v, which is made of
    eighths (at most 2^-12 of its weight goes to page 0, whose v cancel).  The weights are within 2^-17
    of equal (the fp32 score of at most 58, in log2 units, against the row's maximum)."""
    import ctypes

    from scaled_dot_product_prefill_b200 import _lib

    L, page = 2 ** 28 - 100, 256
    kp, vp = (torch.zeros((2, 1, page, D), dtype=torch.bfloat16) for _ in range(2))
    kp[1], q = 3.5, torch.ones((1, 1, D), dtype=torch.bfloat16)
    vp[0, 0, ::2], vp[0, 0, 1::2] = 1.0, -1.0
    vp[1, 0] = torch.from_numpy(np.random.default_rng(D).integers(0, 9, (page, D)) / 8).to(torch.bfloat16)
    table = torch.zeros((1, -(-L // page)), dtype=torch.int32)
    table[0, -1] = 1
    lens, cu = torch.tensor([L], dtype=torch.int32).cuda(), cumulative([1]).cuda()
    dev = [x.cuda() for x in (q, kp, vp, table)]
    out, lse = torch.full((1, 1, D), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((1, 1), 7.0, device="cuda")
    api.attn_device_status(clear=True)
    st = _lib.load().attn_prefill_packed_paged(
        dev[0].data_ptr(), dev[1].data_ptr(), dev[2].data_ptr(), cu.data_ptr(), dev[3].data_ptr(), lens.data_ptr(), page, 1,
        1, 1, 1, D, D, D, 2, table.shape[1], L, D ** -0.5, 1, 0, None, 0, out.data_ptr(), lse.data_ptr(),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and api.attn_device_status(clear=True) == 0
    n, w = L % page, np.exp(3.5 * D ** 0.5)
    want = f64(vp[1, 0, :n]).sum(0) * w / (n * w + (L - n))
    assert (np.abs(f64(out)[0, 0] - want) <= (2.0 ** -8 + 2.0 ** -16) * want).all()
    want = np.log(n * w + (L - n))
    assert abs(float(lse) - want) <= 2.0 ** -17 + 2.0 ** -22 * (want + 16)


def repeated_pages(q, kp, vp, L, workspace=False):
    """(out, lse) of one sequence of L keys whose page table names the pool's pages over and over, on one SM (without a
    workspace) or split; q [1, 1, D]."""
    import ctypes

    from scaled_dot_product_prefill_b200 import _lib

    num, _, page, D = kp.shape
    table = (torch.arange(-(-L // page), dtype=torch.int32) % num).view(1, -1).cuda()
    lens, cu = torch.tensor([L], dtype=torch.int32).cuda(), cumulative([1]).cuda()
    q, kp, vp = q.cuda(), kp.cuda(), vp.cuda()
    need = api.attn_prefill_packed_workspace_size(1, 1, 1, 1, D, L) if workspace else 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(q, 9.0), torch.full((1, 1), 7.0, device="cuda")
    api.attn_device_status(clear=True)
    st = _lib.load().attn_prefill_packed_paged(
        q.data_ptr(), kp.data_ptr(), vp.data_ptr(), cu.data_ptr(), table.data_ptr(), lens.data_ptr(), page, 1, 1, 1, 1, D, D,
        D, num, table.shape[1], L, D ** -0.5, 1, 0, ws.data_ptr() if workspace else None, need, out.data_ptr(),
        lse.data_ptr(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and api.attn_device_status(clear=True) == 0
    return f64(out)[0, 0], float(lse)


@pytest.mark.parametrize("D", [64, 128])
def test_the_sum_over_many_keys_of_like_weight(D):
    """2^28 keys of equal weight, v 0, 1 or 2 of one sign a column.  A run of 2^16 keys sums to 2^16 v, the runs to
    multiples of that below 2^29: exact in fp32.  The last, shorter run and the sum of the weights round by
    2^-24 each, which no bf16 value of 0, 1 or 2 notices."""
    L = 2 ** 28 - 100
    v = (torch.arange(D) % 5 - 2).to(torch.bfloat16)
    out, lse = repeated_pages(torch.zeros((1, 1, D), dtype=torch.bfloat16), inputs.normal((1, 1, 256, D), 1),
                              v.expand(1, 1, 256, D).contiguous(), L)
    assert np.array_equal(out, f64(v))
    assert abs(lse - np.log(L)) <= 2.0 ** -22 * (np.log(L) + 16)


@pytest.mark.parametrize("D,log2_keys,workspace", [(64, 18, False), (64, 19, False), (64, 22, False), (128, 20, False),
                                                   (128, 22, False), (64, 22, True), (64, 24, True), (128, 24, True)])
def test_values_of_one_sign_lose_nothing_to_the_length(D, log2_keys, workspace):
    """Equal weights (of exactly 1), v in [0, 1): the mean of v.

    The tensor core aligns 16 products with their sum and drops what lies below 2^-25 of it (as measured: a
    product of 1 is lost beside 2^26, not beside 2^25), and its result is an fp32 value.  A run of 2^16 keys so
    loses 2^16 2^-25 of itself and 2^12 2^-23 at most; up to 2^18 keys (here: the part of a split too) are
    one run.  The up to 2^8 runs round by 2^-24 each, the output by 2^-8.  (One run over all keys lost
    2.2 % of 2^22, 35 % of 2^26.)"""
    r = np.random.default_rng(D + log2_keys)
    vp = torch.from_numpy(r.random((64, 1, 256, D))).to(torch.bfloat16)
    out, lse = repeated_pages(torch.zeros((1, 1, D), dtype=torch.bfloat16), inputs.normal((64, 1, 256, D), 1), vp,
                              2 ** log2_keys, workspace)
    want = f64(vp).reshape(-1, D).mean(0)
    part = log2_keys - 4 * workspace
    run = 2.0 ** (part if part <= 18 else 16)
    assert (np.abs(out - want) <= (run * (2.0 ** -25 + 2.0 ** -27) + 2.0 ** -16 + 2.0 ** -8) * want).all()
    want = log2_keys * np.log(2)
    assert abs(lse - want) <= 2.0 ** -22 * (want + 16)


@pytest.mark.parametrize("D,causal,window", [(64, True, 0), (128, True, 0), (64, False, 0), (128, True, 280_000),
                                             (64, True, 66_000)])
def test_runs_of_keys_are_joined(D, causal, window):
    """Rows over two and more runs of 2^16 keys (one run, with the shortest window), with scores whose maximum grows along the keys (and, in the
    third head, falls), without a workspace."""
    import ctypes

    from scaled_dot_product_prefill_b200 import _lib

    Hq, Hkv, lk = 4, 2, [300_000, 130_000]      # (more than 2^18 rows in the buffer)
    cu_q, cu_k = cumulative([3, 200]), cumulative(lk)
    q, k, v = tensors(203, sum(lk), Hq, Hkv, D, 3)
    ramp = torch.cat([torch.arange(n) / n for n in lk])[:, None, None]
    k = (k.float() * torch.cat((0.2 + 2 * ramp, 2 - 1.9 * ramp), 1)).to(torch.bfloat16)
    v = (v.float() + 0.5).to(torch.bfloat16)
    dev = [x.cuda() for x in (q, k, v, cu_q, cu_k)]
    out, lse = torch.empty_like(dev[0]), torch.empty((203, Hq), device="cuda")
    api.attn_device_status(clear=True)
    st = _lib.load().attn_prefill_packed(
        *(x.data_ptr() for x in dev), 2, 203, sum(lk), Hq, Hkv, D, Hq * D, Hkv * D, Hkv * D, Hq * D, D ** -0.5, int(causal),
        window, None, 0, out.data_ptr(), lse.data_ptr(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and api.attn_device_status(clear=True) == 0
    some = [0, 1, 2, 3, 66, 135, 202]           # rows that the definition is evaluated at
    for b, (a, e) in enumerate(zip(cu_k.tolist(), cu_k.tolist()[1:])):
        for i in [x for x in some if cu_q[b] <= x < cu_q[b + 1]]:
            last = e - (int(cu_q[b + 1]) - 1 - i) if causal else e
            first = max(a, last - window) if window else a
            want = packed_attention(f64(q[i:i + 1]), f64(k[first:last]), f64(v[first:last]), [0, 1], [0, last - first],
                                    D ** -0.5)
            assert_packed((out[i:i + 1], lse[i:i + 1]), want, f"row {i}")


@pytest.mark.parametrize("Hq,Hkv,D,page,new,window,split", [
    (8, 2, 128, 16, [9, 9], 1, False), (8, 2, 128, 16, [9, 9], 128, False), (8, 2, 128, 16, [9, 9], 256, True),
    (8, 2, 128, 0, [9, 9], 128, False), (8, 2, 128, 0, [9, 9], 1000, True), (16, 16, 64, 32, [1], 256, False),
    (16, 16, 64, 32, [1], 400, True), (4, 4, 64, 0, [200, 100], 100, False), (8, 2, 128, 64, [9, 9], 2 ** 31 - 1, True)])
def test_only_key_tiles_in_the_window_are_worth_a_split(Hq, Hkv, D, page, new, window, split):
    """Rows that see 3 key tiles at most through their window are not split over a long cache; the workspace shows it."""
    lk = [4000 + 100 * b for b in range(len(new))]
    cu_q, cu_k = cumulative(new), cumulative(lk)
    q = inputs.normal((sum(new), Hq, D), 5)
    need = api.attn_prefill_packed_workspace_size(len(new), sum(new), Hq, Hkv, D, max(lk))
    assert need > 0
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    api.attn_device_status(clear=True)
    if page:
        p = inputs.paged_inputs(len(lk), Hq, Hkv, D, page, seed=9, seq_lens=lk, spare_pages=3, poison=True)
        K, V = gathered(p, lk)
        got = api.attn_prefill_packed_paged(q.cuda(), p.k_pool.cuda(), p.v_pool.cuda(), cu_q.cuda(), p.page_table.cuda(),
                                            p.seq_lens.cuda(), max_seq_len=max(lk), window=window, want_lse=True,
                                            workspace=ws)
    else:
        k, v = inputs.normal((sum(lk), Hkv, D), 6), inputs.normal((sum(lk), Hkv, D), 7)
        K, V = f64(k), f64(v)
        got = api.attn_prefill_packed(q.cuda(), k.cuda(), v.cuda(), cu_q.cuda(), cu_k.cuda(), window=window,
                                      want_lse=True, workspace=ws)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    assert bool((ws != 0xA5).any()) == split
    assert_packed(got, packed_attention(f64(q), K, V, cu_q.tolist(), cu_k.tolist(), D ** -0.5, True, window))


@pytest.mark.parametrize("Hq,Hkv,D,B,Tq,live", [
    (8, 2, 128, 64, 64, {5: (9, 5000), 63: (9, 4100)}),                      # most slots of a decode batch idle
    (32, 8, 128, 64, 2048, {0: (16, 3000), 17: (16, 2000), 40: (16, 1), 41: (1, 700)}),
    (12, 12, 64, 300, 900, {299: (1, 6000), 100: (300, 300), 150: (0, 800)}),
    (4, 1, 64, 2000, 2000, {1999: (3, 2500)}),
])
def test_idle_slots_beside_long_live_sequences(Hq, Hkv, D, B, Tq, live):
    """A batch and buffers for the largest step, of which a few sequences are live; the rest has no tokens, and half of
    it no cache either."""
    new, lens = [0] * B, [7 * (b % 2) for b in range(B)]
    for b, (n, L) in live.items():
        new[b], lens[b] = n, L
    p = inputs.paged_inputs(B, Hq, Hkv, D, 16, seed=B, seq_lens=lens, spare_pages=3, poison=True)
    q = inputs.normal((Tq, Hq, D), 3)
    q[sum(new):] = float("nan")
    cu = cumulative(new)
    out, lse = torch.full((Tq, Hq, D), 3.5, dtype=torch.bfloat16, device="cuda"), torch.full((Tq, Hq), -7.25, device="cuda")
    api.attn_device_status(clear=True)
    api.attn_prefill_packed_paged(q.cuda(), p.k_pool.cuda(), p.v_pool.cuda(), cu.cuda(), p.page_table.cuda(),
                                  p.seq_lens.cuda(), max_seq_len=max(lens), out=out, lse=lse)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    K, V = gathered(p, lens)
    assert_packed((out, lse), packed_attention(f64(q), K, V, cu.tolist(), cumulative(lens).tolist(), D ** -0.5))
    assert (out[sum(new):] == 3.5).all() and (lse[sum(new):] == -7.25).all()
