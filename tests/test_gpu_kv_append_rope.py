"""GPU tests of the rotating append (attn_kv_append_rope, attn_kv_append_rope_fp8) and of the packed serving loop."""
import numpy as np
import pytest
import torch

from oracle import fp8, sdpa
from packed_oracle import U, assert_packed, cos_sin_table, cumulative, f64, packed_attention, rotate
from scaled_dot_product_prefill_b200 import PagePool, api, inputs

pytestmark = pytest.mark.gpu

# Hq, Hkv, D, rot, page, new tokens, cached tokens (new ones included), interleaved
CASES = [
    (32, 8, 128, 128, 16, [1] * 5, [1, 16, 17, 300, 1000], False),       # one decode step
    (12, 12, 64, 64, 16, [1, 1, 1], [5, 33, 64], True),
    (8, 2, 128, 64, 32, [7, 0, 130, 1], [7, 40, 300, 1], False),         # half of each head turns
    (8, 2, 128, 32, 64, [60, 3], [200, 64], True),
    (4, 1, 64, 16, 8, [9, 20], [9, 21], False),
    (6, 2, 96, 96, 16, [11, 40], [50, 40], True),                        # 6 lanes a row: two lanes of a warp idle
    (3, 1, 256, 256, 16, [5, 18], [100, 18], False),
    (2, 2, 512, 128, 24, [3, 30], [3, 64], True),
    (5, 5, 16, 16, 16, [33, 2], [40, 2], False),
    (4, 2, 80, 0, 16, [10, 5], [30, 5], False),                          # no rotation: a packed append
    (0, 4, 128, 128, 16, [10, 1, 5], [30, 1, 5], False),                 # no q
    (16, 4, 128, 128, 256, [700, 900], [1000, 900], False),              # several rows per warp
    (16, 4, 64, 64, 128, [700, 901], [1000, 901], True),
]


def make(case, seed, fp8_scales=None):
    Hq, Hkv, D, rot, page, new, lens, inter = case
    T = sum(new)
    q = inputs.normal((T, Hq, D), seed) if Hq else None
    k, v = inputs.normal((T, Hkv, D), seed + 1), inputs.normal((T, Hkv, D), seed + 2)
    kw = dict(seq_lens=lens, spare_pages=3)
    if fp8_scales:
        p = inputs.paged_inputs_fp8(len(lens), 1, Hkv, D, page, seed, k_scale=fp8_scales[0], v_scale=fp8_scales[1], **kw)
    else:
        p = inputs.paged_inputs(len(lens), 1, Hkv, D, page, seed, poison=True, **kw)
    return q, k, v, p, cos_sin_table(max(lens), rot) if rot else None


def positions(new, lens):
    """(row, sequence, position) of every new token that has one."""
    row = 0
    for b, (n, L) in enumerate(zip(new, lens)):
        for i in range(n):
            if L - n + i >= 0:
                yield row, b, L - n + i
            row += 1


def expected(case, q, k, v, p, table):
    """Rotated q and k (values, bounds of their terms) by row, and the pool slots of each row."""
    Hq, Hkv, D, rot, page, new, lens, inter = case
    at = list(positions(new, lens))
    rows = np.array([r for r, _, _ in at])
    angles = f64(table)[[x for _, _, x in at]] if rot else np.zeros((len(at), 0))
    turned = {}
    for name, x in (("q", q), ("k", k)):
        if x is not None:
            turned[name] = rotate(f64(x)[rows], angles, inter) if rot else (f64(x)[rows], np.zeros((len(at),) + x.shape[1:]))
    pt = p.page_table.numpy()
    phys = np.array([pt[b, x // page] for _, b, x in at])
    slot = np.array([x % page for _, _, x in at])
    return rows, turned, phys, slot


def close(got, value, mag, what):
    """bf16 results: half a step of the value, and 2^-23 of the terms for the fp32 products and sum."""
    off = np.abs(got - value) - (U * np.abs(value) + 2.0 ** -23 * (1 + U) * mag)
    assert (off <= 0).all(), f"{what}: {off.max():.3e} over the bound"


def bits(t):
    return t.cpu().view(torch.int16).numpy()


def call(q, k, v, kp, vp, table, p, cu, **kw):
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    api.attn_device_status(clear=True)
    scales = {n: kw.pop(n) for n in ("k_scale", "v_scale") if n in kw}
    fn = api.attn_kv_append_rope_fp8 if scales else api.attn_kv_append_rope
    got = fn(c(q), c(k), c(v), kp, vp, c(table), p.page_table.cuda(), p.seq_lens.cuda(), cu_seqlens=c(cu), **scales, **kw)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    return got


@pytest.mark.parametrize("with_k_out", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
def test_rotating_append(case, with_k_out):
    Hq, Hkv, D, rot, page, new, lens, inter = case
    q, k, v, p, table = make(case, seed=sum(lens) + D)
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    k_out = torch.full(k.shape, 7.0, dtype=torch.bfloat16, device="cuda") if with_k_out else None
    same = len(set(new)) == 1
    q_out = call(q, k, v, kp, vp, table, p, None if same else cumulative(new), interleaved=inter, k_out=k_out)
    rows, turned, phys, slot = expected(case, q, k, v, p, table)
    if Hq:
        close(f64(q_out)[rows], *turned["q"], "q_out")
    else:
        assert q_out is None
    close(f64(kp)[phys, :, slot], *turned["k"], "k in the pool")
    if with_k_out:
        # the same values go to both places
        assert np.array_equal(bits(k_out)[rows], bits(kp)[phys, :, slot])
    want_v = bits(p.v_pool).copy()
    want_v[phys, :, slot] = bits(v)[rows]
    assert np.array_equal(bits(vp), want_v)
    # columns that do not turn are kept bit for bit, and so is every slot of no new token
    want_k = bits(p.k_pool).copy()
    want_k[phys, :, slot] = bits(kp)[phys, :, slot]
    want_k[phys, :, slot, rot:] = bits(k)[rows][..., rot:]
    assert np.array_equal(bits(kp), want_k)


@pytest.mark.parametrize("case", [CASES[i] for i in (0, 1, 2, 3, 5, 7, 9, 10, 11)], ids=str)
def test_rotating_append_into_an_8_bit_cache(case):
    Hq, Hkv, D, rot, page, new, lens, inter = case
    ks, vs = 0.013, 0.004     # v saturates now and then
    q, k, v, p, table = make(case, seed=sum(lens) + D, fp8_scales=(ks, vs))
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    q_out = call(q, k, v, kp, vp, table, p, cumulative(new), interleaved=inter, k_scale=ks, v_scale=vs)
    rows, turned, phys, slot = expected(case, q, k, v, p, table)
    if Hq:
        close(f64(q_out)[rows], *turned["q"], "q_out")
    # the code nearest to value / scale: half an E4M3 step (2^-4 of it, 2^-10 among subnormals), more by what the
    # fp32 value and its product with 1 / scale may be off (3 roundings of 2^-24 each, and the terms' 2^-23)
    value, mag = turned["k"]
    x, err = value / ks, (2.0 ** -23 * mag + 2.0 ** -22 * np.abs(value)) / ks
    got = fp8.e4m3_value(kp.cpu())[phys, :, slot]
    near = np.clip(x, -448, 448)
    off = np.abs(got - near) - (np.maximum(np.abs(near) * 2.0 ** -4, 2.0 ** -10) + err * (1 + 2.0 ** -4))
    assert (off <= 0).all(), off.max()
    # v, and the columns that do not turn, are encoded exactly as attn_kv_append_fp8 encodes
    want_v = p.v_pool.numpy().copy()
    want_v[phys, :, slot] = fp8.quantize(v, vs)[rows]
    assert np.array_equal(vp.cpu().numpy(), want_v)
    want_k = p.k_pool.numpy().copy()
    want_k[phys, :, slot] = kp.cpu().numpy()[phys, :, slot]
    want_k[phys, :, slot, rot:] = fp8.quantize(k, ks)[rows][..., rot:]
    assert np.array_equal(kp.cpu().numpy(), want_k)


MANY = [
    # as CASES, with so many tokens that a warp takes 4 steps of a token's rows: 1 to 4 warps a token, the last not full
    (5, 5, 16, 16, 16, [2600], [2600], False),         # 15 rows, 32 a step: one step in all
    (40, 20, 16, 16, 32, [1900, 700], [2000, 700], True),
    (6, 2, 96, 96, 16, [900, 400], [950, 400], True),
    (4, 2, 80, 0, 16, [1500], [1500], False),
    (3, 1, 256, 256, 16, [1000], [1100], False),
    (7, 3, 256, 128, 64, [300, 1, 400], [301, 77, 400], True),
    (2, 2, 512, 128, 24, [200, 300], [200, 364], True),
    (9, 2, 512, 512, 16, [250], [250], False),
]


@pytest.mark.parametrize("fp8_scales", [None, (0.013, 0.004)], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", MANY, ids=[str(c) for c in MANY])
def test_rotating_append_of_many_tokens_at_any_head_dim(case, fp8_scales):
    Hq, Hkv, D, rot, page, new, lens, inter = case
    assert sum(new) * -(-(Hq + 2 * Hkv) // (512 // D)) > 148 * 16      # steps of all tokens: more than 16 an SM
    q, k, v, p, table = make(case, seed=sum(lens) + D, fp8_scales=fp8_scales)
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    scales = dict(zip(("k_scale", "v_scale"), fp8_scales)) if fp8_scales else {}
    k_out = torch.full(k.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    q_out = call(q, k, v, kp, vp, table, p, cumulative(new), interleaved=inter, k_out=k_out, **scales)
    rows, turned, phys, slot = expected(case, q, k, v, p, table)
    assert len(rows) == sum(new)
    close(f64(q_out)[rows], *turned["q"], "q_out")
    close(f64(k_out)[rows], *turned["k"], "k_out")
    kept = lambda pool: bits(pool) if not fp8_scales else pool.cpu().numpy()  # noqa: E731
    stored = lambda x, scale: bits(x) if not fp8_scales else fp8.quantize(x, scale)  # noqa: E731
    want_v = kept(p.v_pool).copy()
    want_v[phys, :, slot] = stored(v, fp8_scales and fp8_scales[1])[rows]
    assert np.array_equal(kept(vp), want_v)
    got_k = kept(kp)[phys, :, slot]
    if fp8_scales:   # the bound of test_rotating_append_into_an_8_bit_cache
        ks, (value, mag) = fp8_scales[0], turned["k"]
        near, err = np.clip(value / ks, -448, 448), (2.0 ** -23 * mag + 2.0 ** -22 * np.abs(value)) / ks
        off = np.abs(fp8.e4m3_value(kp.cpu())[phys, :, slot] - near)
        assert (off <= np.maximum(np.abs(near) * 2.0 ** -4, 2.0 ** -10) + err * (1 + 2.0 ** -4)).all()
    else:
        assert np.array_equal(got_k, bits(k_out)[rows])
    want_k = kept(p.k_pool).copy()
    want_k[phys, :, slot] = got_k
    want_k[phys, :, slot, rot:] = stored(k, fp8_scales and fp8_scales[0])[rows][..., rot:]
    assert np.array_equal(kept(kp), want_k)


@pytest.mark.parametrize("inter", [False, True])
def test_in_place_on_slices_of_a_fused_projection(inter):
    Hq, Hkv, D, page, new, lens = 8, 2, 128, 16, [40, 3, 90], [100, 3, 90]
    T = sum(new)
    host = inputs.normal((T, (Hq + 2 * Hkv) * D + 16), 9)
    cut = lambda x, a, h: x[:, a:a + h * D].view(T, h, D)  # noqa: E731
    p = inputs.paged_inputs(3, 1, Hkv, D, page, 4, seq_lens=lens)
    table = cos_sin_table(200, D)
    parts = [(0, Hq), (Hq * D, Hkv), ((Hq + Hkv) * D, Hkv)]
    q, k, v = (cut(host, a, h).contiguous() for a, h in parts)
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    k_out = torch.empty_like(k.cuda())
    q_out = call(q, k, v, kp, vp, table, p, cumulative(new), interleaved=inter, k_out=k_out)
    fused = host.cuda()
    kp2, vp2 = p.k_pool.cuda(), p.v_pool.cuda()
    fq, fk, fv = (cut(fused, a, h) for a, h in parts)
    back = call(fq, fk, fv, kp2, vp2, table, p, cumulative(new), interleaved=inter, q_out=fq, k_out=fk)
    assert back.data_ptr() == fq.data_ptr()
    assert torch.equal(fq, q_out) and torch.equal(fk, k_out) and torch.equal(fv.cpu(), v)
    assert torch.equal(fused[:, (Hq + 2 * Hkv) * D:].cpu(), host[:, (Hq + 2 * Hkv) * D:])
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2)


def test_without_rotation_it_is_the_plain_append():
    B, Hkv, S, D, page, lens = 3, 4, 50, 128, 16, [50, 200, 77]
    p = inputs.paged_inputs(B, 1, Hkv, D, page, 6, seq_lens=lens, poison=True)
    k, v = inputs.normal((B, Hkv, S, D), 1), inputs.normal((B, Hkv, S, D), 2)
    rows = lambda x: x.transpose(1, 2).reshape(B * S, Hkv, D).contiguous()  # noqa: E731
    kp, vp, kp2, vp2 = p.k_pool.cuda(), p.v_pool.cuda(), p.k_pool.cuda(), p.v_pool.cuda()
    api.attn_kv_append(k.cuda(), v.cuda(), kp, vp, p.page_table.cuda(), p.seq_lens.cuda())
    call(None, rows(k), rows(v), kp2, vp2, None, p, None)
    assert np.array_equal(bits(kp), bits(kp2)) and np.array_equal(bits(vp), bits(vp2))


def test_rows_of_no_sequence_and_tokens_without_a_position_are_left_alone():
    Hq, Hkv, D, page = 4, 2, 64, 16
    new, lens, front, back = [6, 10, 4], [20, 7, 4], 5, 90       # sequence 1: the cache is shorter than its chunk
    T = front + sum(new) + back
    q, k, v = inputs.normal((T, Hq, D), 1), inputs.normal((T, Hkv, D), 2), inputs.normal((T, Hkv, D), 3)
    p = inputs.paged_inputs(3, 1, Hkv, D, page, 4, seq_lens=lens, poison=True)
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    q_out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    table = cos_sin_table(64, D)
    call(q, k, v, kp, vp, table, p, cumulative(new, front), q_out=q_out, k_out=k_out)
    case = (Hq, Hkv, D, D, page, new, lens, False)
    inner = slice(front, front + sum(new))
    rows, turned, phys, slot = expected(case, q[inner], k[inner], v[inner], p, table)
    assert len(rows) == 6 + 7 + 4
    close(f64(q_out)[inner][rows], *turned["q"], "q_out")
    left = np.ones(T, bool)
    left[rows + front] = False
    assert (f64(q_out)[left] == 7).all() and (f64(k_out)[left] == 7).all()
    want = bits(p.v_pool).copy()
    want[phys, :, slot] = bits(v)[inner][rows]
    assert np.array_equal(bits(vp), want)


def test_positions_behind_the_table_and_bad_pages_are_reported_and_skipped():
    Hq, Hkv, D, page, new, lens = 4, 2, 64, 16, [40, 40], [40, 40]
    q, k, v = inputs.normal((80, Hq, D), 1), inputs.normal((80, Hkv, D), 2), inputs.normal((80, Hkv, D), 3)
    p = inputs.paged_inputs(2, 1, Hkv, D, page, 4, seq_lens=lens)
    c = lambda x: x.cuda()  # noqa: E731
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    q_out = torch.full((80, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    api.attn_device_status(clear=True)
    api.attn_kv_append_rope(c(q), c(k), c(v), kp, vp, c(cos_sin_table(30, D)), c(p.page_table), c(p.seq_lens),
                            q_out=q_out)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 5
    assert (q_out[30:40] == 7).all() and (q_out[70:] == 7).all() and not (q_out[:30] == 7).all()
    table = p.page_table.numpy()
    last = table[:, 2]                                  # positions 32..39 have no angles: their slots are kept
    assert np.array_equal(bits(vp)[last], bits(p.v_pool)[last])
    # a bad page: the pools are left alone, q is rotated all the same
    bad = p.page_table.clone()
    bad[0, 1], bad[1, 2] = p.num_pages, -1
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    good_q = api.attn_kv_append_rope(c(q), c(k), c(v), p.k_pool.cuda(), p.v_pool.cuda(), c(cos_sin_table(40, D)),
                                     c(p.page_table), c(p.seq_lens))
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    got_q = api.attn_kv_append_rope(c(q), c(k), c(v), kp, vp, c(cos_sin_table(40, D)), c(bad), c(p.seq_lens))
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 5
    assert torch.equal(got_q, good_q)
    for page_id in (table[0, 1], table[1, 2]):
        assert np.array_equal(bits(kp)[page_id], bits(p.k_pool)[page_id])
    # a page table too short for the sequence
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    api.attn_kv_append_rope(c(q), c(k), c(v), kp, vp, c(cos_sin_table(40, D)), c(p.page_table[:, :2].contiguous()),
                            c(p.seq_lens))
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 5
    assert np.array_equal(bits(vp)[last], bits(p.v_pool)[last])


@pytest.mark.parametrize("B", [1, 31, 32, 33, 500, 1100])
def test_the_sequence_of_a_row_is_found_among_many(B):
    """Sequences of 0 to 3 tokens, so that every boundary is met; v's copies show where each row went."""
    new = np.random.default_rng(B).integers(0, 4, B)
    new[-1] = 3
    lens = new + np.arange(B) % 5
    T = int(new.sum())
    p = inputs.paged_inputs(B, 1, 1, 16, 8, 5, seq_lens=lens.tolist(), max_pages=2)
    k, v = inputs.normal((T, 1, 16), 1), inputs.normal((T, 1, 16), 2)
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    call(None, k, v, kp, vp, None, p, cumulative(new))
    rows, _, phys, slot = expected((0, 1, 16, 0, 8, new.tolist(), lens.tolist(), False), None, k, v, p, None)
    for got, pool, x in ((kp, p.k_pool, k), (vp, p.v_pool, v)):
        want = bits(pool).copy()
        want[phys, :, slot] = bits(x)[rows]
        assert np.array_equal(bits(got), want)


@pytest.mark.parametrize("cu", [[0, 50, 20, 80], [0, 30, 60, 4000], [-7, 30, 60, 80], [0, 2 ** 31 - 1, 5, -2 ** 31]])
def test_malformed_cumulative_lengths_stay_in_the_buffers(cu):
    Hkv, D, page = 2, 64, 16
    p = inputs.paged_inputs(3, 1, Hkv, D, page, 4, seq_lens=[100, 100, 100])
    k, v = inputs.normal((80, Hkv, D), 2), inputs.normal((80, Hkv, D), 3)
    big = torch.full((p.num_pages + 20, Hkv, page, D), 5.0, dtype=torch.bfloat16, device="cuda")
    kp = big[10:10 + p.num_pages]
    vp = torch.zeros_like(kp)
    out = torch.full((300, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda")
    api.attn_kv_append_rope(None, k.cuda(), v.cuda(), kp, vp, cos_sin_table(100, D).cuda(), p.page_table.cuda(),
                            p.seq_lens.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                            k_out=out[100:180])
    torch.cuda.synchronize()
    api.attn_device_status(clear=True)
    assert (big[:10] == 5).all() and (big[10 + p.num_pages:] == 5).all()
    assert (out[:100] == 9).all() and (out[180:] == 9).all()


def decreasing_among(B, at):
    """Cumulative lengths of B sequences of 2 tokens; the one that ends sequence `at` is 3 lower than it was."""
    cu = list(range(0, 2 * B + 1, 2))
    cu[at + 1] -= 3
    return cu


@pytest.mark.parametrize("cu", [
    [0, 30, 60, 85], [0, 30, 60, 81], [0, 30, 60, 4000], [0, 30, 80, 85],       # past the 80 rows, by a little or wholly
    [0, 85, 90, 95], [81, 90, 95, 99], [-7, 30, 60, 80], [-3, 0, 40, 80], [-9, -5, 30, 80],
    [0, 50, 20, 80], [0, 2 ** 31 - 1, 5, -2 ** 31], [0, 30, 60, 2 ** 31 - 1],
    decreasing_among(40, 17), decreasing_among(40, 33), decreasing_among(40, 39)], ids=lambda cu: str(cu[:4]) + f"x{len(cu) - 1}")
def test_malformed_cumulative_lengths_are_reported_and_write_no_wrong_slot(cu):
    """Every malformed array is reported, and a row goes to the slot of a sequence that holds it within the
    buffer, or nowhere."""
    T, Hq, Hkv, D, page, B = 80, 4, 2, 64, 16, len(cu) - 1
    lens = [100 + b % 3 for b in range(B)]
    p = inputs.paged_inputs(B, 1, Hkv, D, page, 4, seq_lens=lens)
    q, k, v = inputs.normal((T, Hq, D), 1), inputs.normal((T, Hkv, D), 2), inputs.normal((T, Hkv, D), 3)
    kp, vp = p.k_pool.cuda(), p.v_pool.cuda()
    q_out, k_out = (torch.full((T, h, D), 7.0, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
    api.attn_device_status(clear=True)
    api.attn_kv_append_rope(q.cuda(), k.cuda(), v.cuda(), kp, vp, cos_sin_table(110, D).cuda(), p.page_table.cuda(),
                            p.seq_lens.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                            q_out=q_out, k_out=k_out)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 5
    # where each row may have gone
    slots, held = {}, np.zeros(T, bool)
    for b in range(B):
        if 0 <= cu[b] <= cu[b + 1] <= T:
            for t in range(cu[b], cu[b + 1]):
                x, held[t] = lens[b] - cu[b + 1] + t, True
                slots.setdefault((int(p.page_table[b, x // page]), x % page), set()).add(t)
    before, after = bits(p.v_pool), bits(vp)
    for pg, s in np.argwhere((before != after).any((1, 3))):
        assert any(np.array_equal(after[pg, :, s], bits(v)[t]) for t in slots.get((pg, s), ())), (pg, s)
    assert (q_out.cpu()[~held] == 7).all() and (k_out.cpu()[~held] == 7).all()
    # rows of one sequence alone, which none of the malformed ones claims, are written
    claims = np.zeros(T, int)
    for b in range(B):
        lo, hi = sorted((min(max(cu[b], 0), T), min(max(cu[b + 1], 0), T)))
        claims[lo:hi] += 1
    for (pg, s), rows in slots.items():
        for t in rows:
            if claims[t] == 1:
                assert np.array_equal(after[pg, :, s], bits(v)[t]), t


def test_far_positions_take_their_angles_from_the_table():
    """The last positions of a long cache: the pages in between are not touched, the angles are the table's."""
    Hq, Hkv, D, page, L = 4, 1, 64, 256, 1_000_003
    pages = -(-L // page)
    table = cos_sin_table(L, 64)
    pt = torch.full((1, pages), -1, dtype=torch.int32)
    pt[0, -1] = 2
    q, k, v = inputs.normal((2, Hq, D), 1), inputs.normal((2, Hkv, D), 2), inputs.normal((2, Hkv, D), 3)
    kp, vp = (torch.zeros((4, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    api.attn_device_status(clear=True)
    q_out = api.attn_kv_append_rope(q.cuda(), k.cuda(), v.cuda(), kp, vp, table.cuda(), pt.cuda(),
                                    torch.tensor([L], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    close(f64(q_out), *rotate(f64(q), f64(table)[L - 2:], False), "q_out")
    at = [(L - 2) % page, (L - 1) % page]
    close(f64(kp)[2][:, at].transpose(1, 0, 2), *rotate(f64(k), f64(table)[L - 2:], False), "k")
    assert torch.equal(vp[2][:, at].transpose(0, 1).cpu(), v)


def test_pools_whose_offsets_pass_32_bits():
    """Slots behind element 2^31 of a pool."""
    Hkv, D, page = 8, 128, 256
    num = 2 ** 31 // (Hkv * page * D) + 3
    kp = torch.zeros((num, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k, v = inputs.normal((40, Hkv, D), 2), inputs.normal((40, Hkv, D), 3)
    q = inputs.normal((40, 16, D), 4)
    pt = torch.tensor([[num - 1, 0], [num - 2, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 256], dtype=torch.int32, device="cuda")
    table = cos_sin_table(256, D)
    q_out = api.attn_kv_append_rope(q.cuda(), k.cuda(), v.cuda(), kp, vp, table.cuda(), pt, lens)
    assert torch.equal(vp[num - 1, :, :20].transpose(0, 1).cpu(), v[:20])
    assert torch.equal(vp[num - 2, :, 236:].transpose(0, 1).cpu(), v[20:])
    # and the chunk's attention reads them back from there
    kp[num - 2, :, :236] = 0.5
    vp[num - 2, :, :236] = 0.25
    cu = cumulative([20, 20])
    got = api.attn_prefill_packed_paged(q_out, kp, vp, cu.cuda(), pt, lens, max_seq_len=256, want_lse=True)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    K = np.concatenate([f64(kp[num - 1, :, :20]).transpose(1, 0, 2), f64(kp[num - 2]).transpose(1, 0, 2)])
    V = np.concatenate([f64(vp[num - 1, :, :20]).transpose(1, 0, 2), f64(vp[num - 2]).transpose(1, 0, 2)])
    assert_packed(got, packed_attention(f64(q_out), K, V, cu.tolist(), [0, 20, 276], D ** -0.5))


def test_the_packed_serving_loop():
    """Fused projections of packed prompts: rotate and append, prefill in chunks of unlike lengths over the pages,
    then decode steps; every output against the definition on the cache's own contents, and the whole
    prompt's chunked result against its packed prefill in one call."""
    Hq, Hkv, D, page, scale = 8, 2, 128, 16, 128 ** -0.5
    prompts, max_seqs, max_pages = [150, 1, 70, 260], 4, 24
    pool = PagePool(60, page, max_seqs, max_pages)
    kp = torch.full((60, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    table, lens = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((max_seqs, max_pages), (max_seqs,)))
    angles = cos_sin_table(max_pages * page, D).cuda()
    whole = [inputs.normal((n + 8, (Hq + 2 * Hkv) * D), 100 + i) for i, n in enumerate(prompts)]
    cut = lambda x, a, h: x[:, a * D:(a + h) * D].view(x.shape[0], h, D)  # noqa: E731

    def cached(upto):
        t, _ = pool.export()
        return [np.concatenate([sdpa.gather_pages(p.cpu(), t[s].numpy(), n, page) for s, n in enumerate(upto)])
                for p in (kp, vp)]

    done, outs = [0] * 4, [[] for _ in prompts]
    api.attn_device_status(clear=True)
    while done != prompts:
        take = [min(n - d, c) for n, d, c in zip(prompts, done, (96, 5, 33, 130))]
        x = torch.cat([w[d:d + c] for w, d, c in zip(whole, done, take)]).cuda()
        done = [d + c for d, c in zip(done, take)]
        for s, d in enumerate(done):
            pool.resize(s, d)
        pool.upload(table, lens)
        cu = cumulative(take)
        q = cut(x, 0, Hq)
        api.attn_kv_append_rope(q, cut(x, Hq, Hkv), cut(x, Hq + Hkv, Hkv), kp, vp, angles, table, lens,
                                cu_seqlens=cu.cuda(), q_out=q)
        got = api.attn_prefill_packed_paged(q, kp, vp, cu.cuda(), table, lens, max_seq_len=max(done), want_lse=True)
        torch.cuda.synchronize()
        assert api.attn_device_status(clear=True) == 0
        K, V = cached(done)
        assert_packed(got, packed_attention(f64(q), K, V, cu.tolist(), cumulative(done).tolist(), scale), str(done))
        for s, c in enumerate(take):
            outs[s].append(got[0][int(cu[s]):int(cu[s]) + c])
    # the prompts in one packed call on the rotated keys kept beside the cache
    x = torch.cat([w[:n] for w, n in zip(whole, prompts)]).cuda()
    q, k, v = cut(x, 0, Hq), cut(x, Hq, Hkv), cut(x, Hq + Hkv, Hkv)
    cu = cumulative(prompts).cuda()
    api.attn_kv_append_rope(q, k, v, torch.empty_like(kp), torch.empty_like(vp), angles, table, lens, cu_seqlens=cu,
                            q_out=q, k_out=k)
    one = api.attn_prefill_packed(q, k, v, cu)
    K, V = cached(prompts)
    want = packed_attention(f64(q), K, V, cu.tolist(), cu.tolist(), scale)
    assert_packed((one, None), want, "one call")
    assert_packed((torch.cat([torch.cat(o) for o in outs]), None), want, "in chunks")
    # decode steps
    for step in range(3):
        for s in range(4):
            pool.resize(s, prompts[s] + step + 1)
        pool.upload(table, lens)
        x = torch.stack([w[n + step] for w, n in zip(whole, prompts)]).cuda()
        q = api.attn_kv_append_rope(cut(x, 0, Hq), cut(x, Hq, Hkv), cut(x, Hq + Hkv, Hkv), kp, vp, angles, table, lens)
        out = api.attn_decode_paged(q, kp, vp, table, lens, max_seq_len=max_pages * page)
        single = api.attn_prefill_packed_paged(q, kp, vp, cumulative([1] * 4).cuda(), table, lens,
                                               max_seq_len=max_pages * page)
        torch.cuda.synchronize()
        assert api.attn_device_status(clear=True) == 0
        now = [n + step + 1 for n in prompts]
        K, V = cached(now)
        want = packed_attention(f64(q), K, V, [0, 1, 2, 3, 4], cumulative(now).tolist(), scale)
        assert_packed((out, None), want, f"decode {step}")
        assert_packed((single, None), want, f"single tokens {step}")


def test_append_and_decode_replay_from_a_graph():
    N, Hq, Hkv, D, page = 3, 8, 2, 64, 16
    lens0 = [5, 16, 100]
    p = inputs.paged_inputs(N, Hq, Hkv, D, page, 7, seq_lens=[x + 16 for x in lens0])
    kp, vp, table = p.k_pool.cuda(), p.v_pool.cuda(), p.page_table.cuda()
    angles = cos_sin_table(200, D)
    q, k, v = (torch.zeros((N, h, D), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    sl = torch.tensor(lens0, dtype=torch.int32, device="cuda")
    qo, out = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(api.attn_decode_paged_workspace_size(N, Hq, D, 128, page), dtype=torch.uint8, device="cuda")
    dev_angles = angles.cuda()

    def step():
        api.attn_kv_append_rope(q, k, v, kp, vp, dev_angles, table, sl, q_out=qo, interleaved=True)
        api.attn_decode_paged(qo, kp, vp, table, sl, max_seq_len=128, workspace=ws, out=out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in range(3):
        for x, seed in ((q, 1), (k, 2), (v, 3)):
            x.copy_(inputs.normal(tuple(x.shape), 10 * t + seed))
        now = [x + 1 + t for x in lens0]
        sl.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert api.attn_device_status(clear=True) == 0
        ang = f64(angles)[[x - 1 for x in now]]
        close(f64(qo), *rotate(f64(q), ang, True), "q")
        K, V = (np.concatenate([sdpa.gather_pages(pool.cpu(), table[b].cpu().numpy(), n, page)
                                for b, n in enumerate(now)]) for pool in (kp, vp))
        last = np.cumsum(now) - 1
        close(K[last], *rotate(f64(k), ang, True), "k")
        assert np.array_equal(V[last], f64(v))
        assert_packed((out, None), packed_attention(f64(qo), K, V, [0, 1, 2, 3], cumulative(now).tolist(), D ** -0.5))
    del g
