"""The attention-side operators on the GPU against their definitions in 64
bits: head norms with rotation, the paged INT8 cache, attention over it."""
import numpy as np
import pytest
import torch

import rotated_int8_quantized_b200 as cr
from kv8_reference import BLOCK, Paged, attention, bits_to_f64, norm_rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def status_word_is_clean():
    cr.load_library().convrot_device_status(None)
    yield


def _randn(*shape, seed=0, outliers=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if outliers:
        x[..., 3::29] *= 8
    return x.bfloat16().to(DEV)


# A value goes through a norm (a sum of dim squares: relative error below (dim / 8 + 8) 2^-24, the root halves it), three
# products and a sum of two in FP32: below 24 roundings of 2^-24 of the row's largest pair, then one rounding to BF16.
def _near_bf16(got, want, scale):
    err = np.abs(bits_to_f64(got) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 24 * 2.0 ** -24 * scale).all(), err.max()


@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (128, 8), (64, 64), (64, 24)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,axes,norm", [(1, 1, 0, 1, True), (13, 5, 1, 3, True), (70, 8, 2, 1, False)])
def test_norm_rope(dim, rot, adjacent, tokens, hq, hk, axes, norm):
    qkv = _randn(tokens, hq + 2 * hk, dim, seed=tokens, outliers=True)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk] if hk else None
    w = (1 + 0.3 * torch.randn(2, dim, generator=torch.Generator().manual_seed(1))).bfloat16().to(DEV) if norm else [None, None]
    table = cr.rope_table(50, rot, 1e4)
    pos = torch.randint(0, 50, (axes, tokens), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    axis = torch.randint(0, axes, (rot // 2,), generator=torch.Generator().manual_seed(3), dtype=torch.uint8) if axes > 1 else None
    rope = cr.Rope(table, adjacent, None if axis is None else axis.to(DEV))
    qo, ko = cr.qk_norm_rope(q, k, w[0], w[1], 1e-5, rope, pos.to(DEV))
    for x, y, wt in ((q, qo, w[0]), (k, ko, w[1])):
        if x is None:
            assert y is None
            continue
        ref = norm_rotate(bits_to_f64(x), None if wt is None else bits_to_f64(wt), 1e-5, table.cpu().numpy().astype(np.float64),
                          pos.numpy(), None if axis is None else axis.numpy(), adjacent)
        _near_bf16(y, ref, np.abs(ref).max(-1, keepdims=True))
    # in place, and the same bits
    cr.QKNormRope(q, k, q, k, w[0], w[1], 1e-5, rope, pos.to(DEV))()
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))


def test_norm_rope_many_heads_take_eight_rows_a_group():
    q, k = _randn(2100, 42, 128), _randn(2100, 42, 128, seed=1)
    table, pos = cr.rope_table(2100, 128, 1e6), torch.arange(2100, dtype=torch.int32, device=DEV)
    w = _randn(128, seed=2)
    qo, ko = cr.qk_norm_rope(q, k, w, None, rope=cr.Rope(table), positions=pos)
    for x, y, wt in ((q, qo, w), (k, ko, None)):
        ref = norm_rotate(bits_to_f64(x), None if wt is None else bits_to_f64(wt), 1e-6, table.cpu().numpy().astype(np.float64),
                          pos.cpu().numpy()[None], None, False)
        _near_bf16(y, ref, np.abs(ref).max(-1, keepdims=True))


def test_single_rows_with_odd_strides():
    """A view's stride along an axis of one means nothing."""
    base = _randn(1, 3, 64)
    q = base.as_strided((1, 3, 64), (5, 64, 1))
    one = base[:, :1].as_strided((1, 1, 64), (7, 3, 1))
    assert torch.equal(cr.qk_norm_rope(q, one)[0], base) and torch.equal(cr.qk_norm_rope(q, one)[1], base[:, :1])
    paged = Paged([40], 3, 64, 16)
    out, _ = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len)
    assert torch.equal(out, cr.attn_kv8(base, paged.cache, paged.table_dev, paged.kv_len)[0])


def _bits(x):
    return x.contiguous().view(torch.int16)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rot", [0, 8, 32])
@pytest.mark.parametrize("adjacent", [False, True])
def test_dims_without_rotation_stay_apart(dim, rot, adjacent):
    """Infinities, NaN and the sign of a zero stay where they are in the dims that nothing turns."""
    q = _randn(5, 3, dim)
    for i, value in enumerate((float("inf"), float("-inf"), float("nan"), -0.0)):
        q[i, 1, dim - 1 - 3 * i] = value
        q[i, 2, rot + 2 * i] = value
    rope = cr.Rope(cr.rope_table(9, rot), adjacent) if rot else None
    pos = torch.arange(5, dtype=torch.int32, device=DEV) if rot else None
    out, _ = cr.qk_norm_rope(q, rope=rope, positions=pos)
    x, y = q[..., rot:], out[..., rot:]
    assert torch.equal(x.isnan(), y.isnan()) and torch.equal(_bits(x)[~x.isnan()], _bits(y)[~x.isnan()])
    if rot:
        clean = q.clone()
        clean[..., rot:] = 1
        assert torch.equal(out[..., :rot], cr.qk_norm_rope(clean, rope=rope, positions=pos)[0][..., :rot])
    # normalised by an infinite mean: zeros, and NaN where the infinity was
    w = _randn(dim, seed=1)
    out, _ = cr.qk_norm_rope(q[:2], None, w, rope=rope, positions=None if pos is None else pos[:2])
    for i in range(2):
        for h, d in ((1, dim - 1 - 3 * i), (2, rot + 2 * i)):
            assert out[i, h].isnan().nonzero().flatten().tolist() == [d]
            assert (out[i, h].nan_to_num() == 0).all()


def test_norm_only_and_broadcast_input():
    q = _randn(1, 1, 64).expand(9, 3, 64)
    w = _randn(64, seed=2)
    qo, _ = cr.qk_norm_rope(q, None, w)
    ref = norm_rotate(bits_to_f64(q), bits_to_f64(w), 1e-6, None, None, None, False)
    _near_bf16(qo, ref, np.abs(ref).max(-1, keepdims=True))


def test_positions_outside_the_table_give_zero_rows():
    q = _randn(4, 2, 64)
    rope = cr.Rope(cr.rope_table(10, 64))
    pos = torch.tensor([0, 10, 9, -1], dtype=torch.int32, device=DEV)
    out, _ = cr.qk_norm_rope(q, None, rope=rope, positions=pos)
    assert out[1].abs().max() == 0 and out[3].abs().max() == 0
    assert torch.equal(out[0], q[0]) and out[2].abs().max() > 0
    with pytest.raises(cr.ConvrotError) as e:
        cr.convrot_device_status()
    assert e.value.status == 1
    cr.convrot_device_status()


# ------------------------------------------------------------------ append
def _append(paged, news, hq, hk, dim, seed, rope=None, w=None, cu="cu", v_scale=1.0, k=None, v=None):
    """Appends `news` tokens to every sequence (lens grow); returns what went in."""
    total = sum(news)
    qkv = _randn(total, hq + 2 * hk, dim, seed=seed, outliers=True)
    q, kk, vv = qkv[:, :hq] if hq else None, qkv[:, hq:hq + hk], qkv[:, hq + hk:] * v_scale
    kk, vv = (kk if k is None else k), (vv if v is None else v)
    old = list(paged.lens)
    paged.lens = [a + b for a, b in zip(old, news)]
    paged.kv_len = torch.tensor(paged.lens, dtype=torch.int32, device=DEV)
    cus = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV) if cu == "cu" else None
    before = [x.clone() for x in (paged.cache.k, paged.cache.v, paged.cache.k_scale, paged.cache.v_scale)]
    out = cr.kv8_append(q, kk, vv, paged.cache, paged.table_dev, paged.kv_len, cus, w, w, 1e-6, rope)
    return q, kk, vv, out, old, before


def _check_append(paged, news, k_ref, v_ref, old, before):
    """Codes and scales of the touched blocks, and that nothing else changed."""
    page = paged.page
    for which, ref in ((0, k_ref), (1, v_ref)):
        codes, scales = (paged.cache.k, paged.cache.v)[which].cpu().numpy(), (paged.cache.k_scale, paged.cache.v_scale)[which].cpu().numpy()
        codes0, scales0 = before[which].cpu().numpy(), before[2 + which].cpu().numpy()
        same, same_s = codes == codes0, (scales == scales0) | (np.isnan(scales) & np.isnan(scales0))
        t = 0
        for b, n in enumerate(news):
            p = old[b]
            while p < old[b] + n:
                off = p % BLOCK
                m = min(BLOCK - off, old[b] + n - p)
                pg, row = int(paged.table[b, p // page]), p % page // BLOCK
                lo = p % page - off
                x = ref[t:t + m]                                         # [m, heads, dim]
                s, c = scales[pg, :, row].astype(np.float64), codes[pg, :, lo + off:lo + off + m].astype(np.float64)
                most = np.abs(x).max((0, 2))
                if off == 0:
                    # amax / 127, the values of x within 24 FP32 roundings
                    assert (np.abs(s - most / 127) <= 32 * 2.0 ** -24 * most / 127).all()
                else:
                    s0 = scales0[pg, :, row].astype(np.float64)
                    j = np.log2(s / s0)
                    assert (j == np.rint(j)).all() and (j >= 0).all()
                    assert (most < 127.5 * s * (1 + 2.0 ** -19)).all()
                    assert ((j == 0) | (most >= 127.5 * s / 2 * (1 - 2.0 ** -19))).all()
                    c0 = codes0[pg, :, lo:lo + off].astype(np.float64)
                    assert np.array_equal(codes[pg, :, lo:lo + off], np.rint(c0 / 2.0 ** j[:, None, None]))
                # half a step, and the FP32 error of x / s (at most 128 * 32 * 2^-24)
                err = np.abs(c * s[:, None, None] - x.transpose(1, 0, 2))
                clamped = np.abs(c) == 127
                assert (err <= s[:, None, None] * np.where(clamped, 0.5 + 2.0 ** -10, 0.5 + 2.0 ** -12)).all()
                same[pg, :, lo:lo + off + m] = True
                same_s[pg, :, row] = True
                p, t = p + m, t + m
        assert same.all() and same_s.all()


@pytest.mark.parametrize("dim,hq,hk,page", [(128, 8, 2, 64), (64, 3, 3, 16), (128, 2, 1, 256)])
@pytest.mark.parametrize("norm", [False, True])
def test_append(dim, hq, hk, page, norm):
    lens, news = [0, 5, 16, 100, 31, 0, 240], [3, 1, 33, 28, 1, 0, 70]
    paged = _roomy(lens, [a + b for a, b in zip(lens, news)], hk, dim, page)
    table = cr.rope_table(400, dim, 1e4)
    w = _randn(dim, seed=9) if norm else None
    q, k, v, out, old, before = _append(paged, news, hq, hk, dim, 4, cr.Rope(table), w)
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(old, news)])
    wt = None if w is None else bits_to_f64(w)
    cs = table.cpu().numpy().astype(np.float64)
    kr = norm_rotate(bits_to_f64(k), wt, 1e-6, cs, pos[None], None, False)
    qr = norm_rotate(bits_to_f64(q), wt, 1e-6, cs, pos[None], None, False)
    _near_bf16(out, qr, np.abs(qr).max(-1, keepdims=True))
    _check_append(paged, news, kr, bits_to_f64(v), old, before)
    # the same call again stores the same
    after = [x.clone() for x in (paged.cache.k, paged.cache.v, paged.cache.k_scale, paged.cache.v_scale)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV)
    cr.kv8_append(q, k, v, paged.cache, paged.table_dev, paged.kv_len, cu, w, w, 1e-6, cr.Rope(table))
    for x, y in zip(after[:2], (paged.cache.k, paged.cache.v)):
        assert torch.equal(x, y)
    for x, y in zip(after[2:], (paged.cache.k_scale, paged.cache.v_scale)):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())
    cr.convrot_device_status()


def _roomy(lens, need, hk, dim, page, seed=0):
    """A cache with pages for `need` tokens of which `lens` are stored."""
    paged = Paged(need, hk, dim, page, seed)
    paged.lens = list(lens)
    paged.kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return paged


@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (128, 8), (64, 64), (64, 24)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("axes", [0, 1, 3])
def test_append_rotations(dim, rot, adjacent, axes):
    """Adjacent pairs, rotation of a part of the head, positions given (axes of them) or the cache's own."""
    hq, hk, page = 5, 2, 32
    lens, news = [0, 5, 16, 100, 0, 40], [3, 1, 33, 28, 0, 7]
    paged = _roomy(lens, [a + b for a, b in zip(lens, news)], hk, dim, page)
    old, total = list(lens), sum(news)
    g = torch.Generator().manual_seed(rot + axes)
    table = cr.rope_table(150, rot, 1e4)
    pos = torch.randint(0, 150, (axes, total), generator=g, dtype=torch.int32) if axes else \
        torch.cat([torch.arange(a, a + n) for a, n in zip(old, news)]).int()[None]
    axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.uint8) if axes > 1 else None
    rope = cr.Rope(table, adjacent, None if axis is None else axis.to(DEV))
    qkv = _randn(total, hq + 2 * hk, dim, seed=dim + rot, outliers=True)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    wq, wk = _randn(dim, seed=8), _randn(dim, seed=9)
    paged.lens = [a + b for a, b in zip(old, news)]
    kv_len = torch.tensor(paged.lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV)
    before = [x.clone() for x in (paged.cache.k, paged.cache.v, paged.cache.k_scale, paged.cache.v_scale)]
    out = cr.kv8_append(q, k, v, paged.cache, paged.table_dev, kv_len, cu, wq, wk, 1e-5, rope, pos.to(DEV) if axes else None)
    cs, ax = table.cpu().numpy().astype(np.float64), None if axis is None else axis.numpy()
    qr, kr = (norm_rotate(bits_to_f64(x), bits_to_f64(w), 1e-5, cs, pos.numpy(), ax, adjacent) for x, w in ((q, wq), (k, wk)))
    _near_bf16(out, qr, np.abs(qr).max(-1, keepdims=True))
    _check_append(paged, news, kr, bits_to_f64(v), old, before)
    cr.convrot_device_status()


def test_append_single_tokens_with_positions_of_three_axes():
    """As a video model's decode step takes them; one of the four slots idle, one with a position outside the table."""
    hq, hk, dim = 4, 1, 64
    paged = _roomy([0, 7, 31, 0], [16, 16, 48, 16], hk, dim, 16)
    q, k, v = (_randn(4, h, dim, seed=h + 1) for h in (hq, hk, hk))
    table = cr.rope_table(40, dim, 1e4)
    axis = (torch.arange(dim // 2) % 3).to(torch.uint8)
    pos = torch.tensor([[3, 9, 11, 5], [0, 39, 2, 5], [7, 1, 40, 5]], dtype=torch.int32)
    kv_len = torch.tensor([1, 8, 32, 0], dtype=torch.int32, device=DEV)
    paged.lens = kv_len.tolist()
    before = [x.clone() for x in (paged.cache.k, paged.cache.v, paged.cache.k_scale, paged.cache.v_scale)]
    out = cr.kv8_append(q, k, v, paged.cache, paged.table_dev, kv_len, rope=cr.Rope(table, True, axis.to(DEV)),
                        positions=pos.to(DEV))
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()
    pos[2, 2] = 0                                            # the row written as zeros, see below
    qr, kr = (norm_rotate(bits_to_f64(x), None, 0, table.cpu().numpy().astype(np.float64), pos.numpy(), axis.numpy(), True)
              for x in (q, k))
    qr[2:], kr[2] = 0, 0
    _near_bf16(out, qr, np.abs(qr).max(-1, keepdims=True))
    _check_append(paged, [1, 1, 1, 0], kr[:3], bits_to_f64(v)[:3], [0, 7, 31, 0], before)


def test_append_rotates_queries_in_place():
    hq, hk, dim, news = 6, 2, 128, [40, 1, 9]
    paged = _roomy([3, 0, 20], [43, 1, 29], hk, dim, 16)
    paged.kv_len = torch.tensor([43, 1, 29], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 40, 41, 50], dtype=torch.int32, device=DEV)
    qkv, w, rope = _randn(50, hq + 2 * hk, dim), _randn(dim, seed=1), cr.Rope(cr.rope_table(50, dim), True)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    rest = qkv[:, hq:].clone()
    want = cr.kv8_append(q, k, v, paged.cache, paged.table_dev, paged.kv_len, cu, w, w, rope=rope)
    stored = [x.clone() for x in (paged.cache.k, paged.cache.v)]
    cr.KV8Append(q, k, v, paged.cache, paged.table_dev, paged.kv_len, q, cu=cu, q_weight=w, k_weight=w, rope=rope)()
    assert torch.equal(q, want) and torch.equal(qkv[:, hq:], rest)
    assert torch.equal(stored[0], paged.cache.k) and torch.equal(stored[1], paged.cache.v)
    cr.convrot_device_status()


def test_append_token_by_token_stays_within_a_step():
    """Sixteen calls fill a block, every token larger than the last: each value ends within one step of its block's
    scale, the bound that doubling gives."""
    hk, dim = 2, 64
    paged = _roomy([0], [40], hk, dim, 16)
    rows_k, rows_v = [], []
    for i in range(40):
        k = _randn(1, hk, dim, seed=100 + i) * float(1.13 ** i)
        v = _randn(1, hk, dim, seed=200 + i) * float(1.5 ** (i % 16) if i < 32 else 0.0)
        rows_k.append(bits_to_f64(k))
        rows_v.append(bits_to_f64(v))
        _append(paged, [1], 0, hk, dim, 0, cu=None, k=k, v=v)
    for which, rows in ((0, rows_k), (1, rows_v)):
        got, x = paged.values(0, which), np.concatenate(rows)
        s = (paged.cache.k_scale, paged.cache.v_scale)[which].cpu().numpy()
        for t in range(40):
            step = s[int(paged.table[0, t // 16]), :, 0][:, None]
            assert (np.abs(got[t] - x[t]) <= step * (1 + 2.0 ** -10)).all()
    assert (paged.values(0, 1)[32:] == 0).all()          # all-zero block: scale 0
    cr.convrot_device_status()


def test_append_ties_go_to_even_and_the_scale_doubles_at_127_and_a_half():
    hk, dim = 1, 64
    row = torch.zeros(64)
    row[:16] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 3.5, 20.5, 21.5, -40.5, 63.5, -127.0, 1.0, 0.25, 126.0])
    x = row.bfloat16().view(1, hk, dim).to(DEV)
    for second, scale in ((127.0, 1.0), (127.5, 2.0), (255.0, 4.0), (254.0, 2.0)):
        paged = _roomy([0], [16], hk, dim, 16)
        _append(paged, [1], 0, hk, dim, 0, cu=None, k=x, v=x)
        page = int(paged.table[0, 0])
        assert float(paged.cache.v_scale[page, 0, 0]) == 1.0
        assert paged.cache.v[page, 0, 0, :16].tolist() == [127, 0, 2, 2, 0, -2, -2, 4, 20, 22, -40, 64, -127, 1, 0, 126]
        y = torch.zeros_like(x)
        y[..., 0] = second
        _append(paged, [1], 0, hk, dim, 0, cu=None, k=x, v=y)
        assert float(paged.cache.v_scale[page, 0, 0]) == scale
        first = np.array([127, 0, 2, 2, 0, -2, -2, 4, 20, 22, -40, 64, -127, 1, 0, 126], dtype=np.float64)
        assert paged.cache.v[page, 0, 0, :16].tolist() == np.rint(first / scale).tolist()
        assert int(paged.cache.v[page, 0, 1, 0]) == min(127, round(second / scale))


def test_append_after_a_block_of_zeros_and_far_larger_values():
    hk, dim = 1, 64
    paged = _roomy([0], [16], hk, dim, 16)
    zero = torch.zeros(1, hk, dim, dtype=torch.bfloat16, device=DEV)
    small, large = _randn(1, hk, dim) * 2.0 ** -60, _randn(1, hk, dim, seed=1) * 2.0 ** 20
    for x in (zero, small, zero, large, small):
        _append(paged, [1], 0, hk, dim, 0, cu=None, k=x, v=x)
    got = paged.values(0, 0)
    s = float(paged.cache.k_scale[int(paged.table[0, 0]), 0, 0])
    assert abs(s - float(large.abs().max()) / 127) <= 2.0 ** -22 * s
    assert (got[[0, 1, 2, 4]] == 0).all() and np.abs(got[3] - bits_to_f64(large)[0]).max() <= s / 2 * (1 + 2.0 ** -10)


def test_append_padding_and_what_it_leaves_alone():
    hk, hq, dim = 2, 4, 64
    paged = _roomy([0, 7, 0], [16, 32, 16], hk, dim, 16)
    # single tokens, the first and last slots idle (kv_len 0)
    q, k, v = (_randn(3, h, dim, seed=h) for h in (hq, hk, hk))
    kv_len = torch.tensor([0, 8, 0], dtype=torch.int32, device=DEV)
    before = paged.cache.k.clone()
    out = cr.kv8_append(q, k, v, paged.cache, paged.table_dev, kv_len, rope=cr.Rope(cr.rope_table(16, 64)))
    assert out[0].abs().max() == 0 and out[2].abs().max() == 0 and out[1].abs().max() > 0
    changed = (paged.cache.k != before).any(-1).any(1)
    page = int(paged.table[1, 0])
    assert changed.nonzero().tolist() in ([[page, r] for r in range(8)], [[page, 7]])
    # rows behind the last sequence stay as they were
    x = torch.full((6, hq, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, 2, 3, 3], dtype=torch.int32, device=DEV)
    q, k, v = (_randn(6, h, dim, seed=h) for h in (hq, hk, hk))
    kv_len = torch.tensor([2, 9, 0], dtype=torch.int32, device=DEV)
    before = paged.cache.v.clone()
    cr.KV8Append(q, k, v, paged.cache, paged.table_dev, kv_len, x, cu=cu)()
    assert (x[3:] == 7).all() and torch.equal(x[:3], q[:3])
    assert (paged.cache.v != before).any(-1).any(1).sum() <= 2 + 9
    cr.convrot_device_status()


def test_append_bad_pages_are_recorded_and_skipped():
    hk, dim = 1, 64
    paged = _roomy([0, 0], [40, 40], hk, dim, 16)
    table = paged.table_dev.clone()
    table[0, 1] = 10 ** 6
    table[1, 0] = -3
    k, v = _randn(80, hk, dim), _randn(80, hk, dim, seed=1)
    cu = torch.tensor([0, 40, 80], dtype=torch.int32, device=DEV)
    kv = torch.tensor([40, 40], dtype=torch.int32, device=DEV)
    before = paged.cache.k.clone()
    cr.kv8_append(None, k, v, paged.cache, table, kv, cu)
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()
    changed = {r for r in (paged.cache.k != before).flatten(1).any(1).nonzero()[:, 0].tolist()}
    assert changed == {int(paged.table[0, 0]), int(paged.table[0, 2]), int(paged.table[1, 1]), int(paged.table[1, 2])}
    # longer than its row of the table
    kv = torch.tensor([table.shape[1] * 16 + 5, 40], dtype=torch.int32, device=DEV)
    cr.kv8_append(None, k, v, paged.cache, paged.table_dev, kv, cu)
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()
    # rows in front of the first sequence
    cr.kv8_append(None, k, v, paged.cache, paged.table_dev, torch.tensor([40, 40], dtype=torch.int32, device=DEV),
                  torch.tensor([32, 40, 80], dtype=torch.int32, device=DEV))
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()
    # cu that is no partition of the rows: recorded, nothing out of bounds
    cr.kv8_append(None, k, v, paged.cache, paged.table_dev, torch.tensor([40, 40], dtype=torch.int32, device=DEV),
                  torch.tensor([0, 90, 200], dtype=torch.int32, device=DEV))
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("dim,hk,page", [(128, 2, 64), (64, 5, 16)])
def test_read(dim, hk, page):
    lens = [1, 0, 37, 130, 64]
    paged = Paged(lens, hk, dim, page)
    back = [1, 0, 20, 130, 1]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(back)]), dtype=torch.int32, device=DEV)
    k, v = cr.kv8_read(paged.cache, paged.table_dev, paged.kv_len, sum(back) + 3, cu)
    for which, got in ((0, k), (1, v)):
        ref = np.concatenate([paged.values(b, which)[n - m:] for b, (n, m) in enumerate(zip(lens, back))])
        # the product in FP32 (2^-24) and its rounding to BF16 (2^-8)
        err = np.abs(bits_to_f64(got)[:sum(back)] - ref)
        assert (err <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref)).all()
        assert (got[sum(back):] == 0).all()                # rows behind: as they were
    only, _ = cr.kv8_read(paged.cache, paged.table_dev, paged.kv_len)
    assert (only[1] == 0).all()                            # an empty sequence's row
    assert torch.equal(only[[0, 2, 3, 4]], k[(cu[1:][[0, 2, 3, 4]] - 1).long()])
    cr.convrot_device_status()
    table = paged.table_dev.clone()
    table[3, 0] = 99
    out = torch.ones(130, hk, dim, dtype=torch.bfloat16, device=DEV)
    cr.KV8Read(paged.cache, table[3:4], paged.kv_len[3:4].clone(), out, None,
               cu=torch.tensor([0, 130], dtype=torch.int32, device=DEV))()
    assert (out[:page] == 0).all() and (out[page:] != 0).any()
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()


# ------------------------------------------------------------------ attention
def _check_attention(paged, q, out, lse, news, causal, scale, rows=None):
    """Every row (or `rows` of them per sequence, the last among them) against the definition.

    The weights are rounded to FP16 (2^-12 of each, and exp2 and the products around it less than that again: 2^-11 of
    sum p|v| in all); a score is off by FP32 roundings of sums of |q k|, at most 2^-20 of the largest, which moves a
    weight and the weights' sum by that much each; the result is rounded to BF16 (2^-8).  lse: the score's error and
    FP32 roundings of a sum of weights and of the logarithm.

    FP16 ends at 2^-24, and a weight (times its value scale) is held as 2^4 of its share of the running maximum, so
    each is off by up to half of 2^-24 / 2^4 of that maximum, which is at most the sequence's largest value scale; a
    code is at most 127 and the weights' sum at least 1: 2^-29 * 127 * tokens * largest scale in all.  (Where a later
    token moves the maximum, a weight already rounded is rounded again: 2^-11 counts both.)"""
    t = 0
    o, z = bits_to_f64(out), lse.cpu().numpy().astype(np.float64)
    qf = bits_to_f64(q)
    for b, n in enumerate(news):
        k, v = paged.values(b, 0), paged.values(b, 1)
        used = paged.table.numpy()[b][:-(-paged.lens[b] // paged.page)]
        lost = 2.0 ** -29 * 127 * paged.lens[b] * np.nanmax(paged.cache.v_scale.cpu().numpy()[used], initial=0)
        pick = range(n) if rows is None or n <= rows else sorted(set(np.linspace(0, n - 1, rows).astype(int)))
        for i in pick:
            # row i alone: a causal row sees len - n + i + 1 tokens
            m = max(0, paged.lens[b] - n + i + 1) if causal else paged.lens[b]
            ref, rl, mag, reach = attention(qf[t + i:t + i + 1], k[:m], v[:m], 1, False, scale)
            err = np.abs(o[t + i] - ref[0])
            tol = 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -11 + 2.0 ** -18 * reach[0][:, None]) * mag[0] + lost
            assert (err <= tol).all(), (b, i, (err - tol).max())
            if m == 0:
                assert (o[t + i] == 0).all() and (z[t + i] == -np.inf).all()
            else:
                assert (np.abs(z[t + i] - rl[0]) <= 2.0 ** -18 * (1 + np.abs(rl[0]) + reach[0])).all()
        t += n


def _attend(lens, news, hq, hk, dim, page, causal=True, scale=None, seed=0, cu=True, q=None, **kw):
    paged = Paged(lens, hk, dim, page, seed)
    q = _randn(sum(news), hq, dim, seed=seed + 1) * 2 if q is None else q
    cus = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV) if cu else None
    out, lse = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, cus, scale, causal)
    cr.convrot_device_status()
    _check_attention(paged, q, out, lse, news, causal, dim ** -0.5 if scale is None else scale, **kw)
    return paged, q, out, lse, cus


LENS = [1, 0, 15, 16, 17, 63, 64, 65, 129, 700]


@pytest.mark.parametrize("dim,hq,hk,page", [(128, 8, 1, 64), (128, 8, 8, 16), (64, 12, 4, 32), (64, 16, 1, 256),
                                            (128, 10, 2, 128), (128, 40, 2, 64), (64, 128, 1, 1024), (128, 100, 1, 16)])
def test_attention_single_tokens(dim, hq, hk, page):
    _attend(LENS, [1] * len(LENS), hq, hk, dim, page, cu=False)


@pytest.mark.parametrize("length", [1, 16, 50, 577, 4099])
def test_attention_one_sequence_is_split(length):
    _attend([length], [1], 16, 2, 128, 16, cu=False)


@pytest.mark.parametrize("dim,hq,hk,page", [(128, 8, 1, 64), (64, 6, 2, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_short_runs(dim, hq, hk, page, causal):
    lens, news = [5, 40, 0, 130, 33, 3], [5, 3, 0, 7, 1, 2]
    _attend(lens, news, hq, hk, dim, page, causal)


@pytest.mark.parametrize("dim,hq,hk,page", [(128, 8, 1, 64), (64, 3, 3, 16), (128, 14, 2, 32)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_prompts(dim, hq, hk, page, causal):
    lens, news = [130, 1, 300, 17, 64], [130, 1, 45, 17, 63]
    _attend(lens, news, hq, hk, dim, page, causal, rows=12)


@pytest.mark.parametrize("dim,hq,hk", [(128, 8, 1), (64, 2, 2), (128, 3, 1)])
def test_attention_a_long_prompt(dim, hq, hk):
    _attend([1111], [1111], hq, hk, dim, 64, rows=9)
    _attend([1500], [777], hq, hk, dim, 64, rows=9, causal=False)


@pytest.mark.parametrize("dim,hq,hk,lens,news", [
    (128, 16, 2, [4000], [24]), (64, 6, 2, [3000, 130, 0, 2500], [60, 130, 0, 1]), (128, 8, 1, [257, 1030], [20, 33]),
    (128, 40, 8, [2049], [13])])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_short_prompts_on_long_contexts(dim, hq, hk, lens, news, causal):
    """Few tile pairs: several CTAs share a pass and another kernel joins them."""
    paged, q, out, lse, cu = _attend(lens, news, hq, hk, dim, 64, causal, rows=9)
    for _ in range(5):
        again, lse2 = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, cu, None, causal)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    bad = q.clone()
    bad[0, 1, 3] = float("nan")
    out2, _ = cr.attn_kv8(bad, paged.cache, paged.table_dev, paged.kv_len, cu, None, causal)
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
    hit[0, 1] = True
    assert out2[hit].isnan().all() and torch.equal(out2[~hit], out[~hit])


def test_attention_mixes_prompts_and_single_tokens():
    _attend([900, 1, 400, 77, 0, 2000], [300, 1, 1, 1, 0, 1], 16, 2, 128, 64, rows=7)


def test_many_sequences():
    """More sequences than lanes or threads: every search and sum over them takes several rounds."""
    g = torch.Generator().manual_seed(3)
    batch, hk, dim = 1100, 1, 64
    lens = torch.randint(0, 40, (batch,), generator=g).tolist()
    news = [min(n, int(r)) for n, r in zip(lens, torch.randint(0, 4, (batch,), generator=g))]
    paged, q, out, lse, cu = _attend(lens, news, 2, hk, dim, 16)
    # all single tokens, 128 rows each: too many for the streaming kernel's rule
    _attend([n + 1 for n in lens[:170]], [1] * 170, 128, 1, 64, 16, cu=False)
    # the same sequences appended to and read back
    old = [n - m for n, m in zip(lens, news)]
    roomy = _roomy(old, lens, hk, dim, 16)
    _, k, v, _, old, before = _append(roomy, news, 0, hk, dim, 5)
    _check_append(roomy, news, bits_to_f64(k), bits_to_f64(v), old, before)
    kb, vb = cr.kv8_read(roomy.cache, roomy.table_dev, roomy.kv_len, sum(news), cu)
    for which, got in ((0, kb), (1, vb)):
        ref = np.concatenate([roomy.values(b, which)[lens[b] - m:] for b, m in enumerate(news)])
        assert (np.abs(bits_to_f64(got) - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref)).all()
    cr.convrot_device_status()


def test_attention_rows_before_the_sequence_see_nothing():
    # more rows than tokens: the first see nothing under a causal mask
    _attend([3, 0, 20], [9, 4, 40], 8, 2, 64, 16)
    _attend([3, 0, 20], [9, 4, 40], 8, 2, 64, 16, causal=False)
    _attend([100, 130], [300, 130], 8, 1, 128, 16, rows=11)


def test_attention_score_ranges():
    """Sharp softmax, scores far from zero, queries over many binades."""
    for factor in (40.0, 2.0 ** -30, 2.0 ** 12):
        q = _randn(3, 8, 128) * factor
        _attend([70, 300, 1], [1, 1, 1], 8, 1, 128, 16, cu=False, q=q)
    q = _randn(200, 8, 128)
    q[..., ::2] *= 2.0 ** -12
    q[..., 5] *= 64
    _attend([300], [200], 8, 1, 128, 64, q=q, rows=9)
    q[3] = 0
    _attend([300], [200], 8, 1, 128, 64, q=q, scale=3.0, rows=9)


def test_attention_value_scales_over_many_binades():
    lens = [200, 300]
    for news in ([1, 1], [190, 250]):
        paged = Paged(lens, 1, 128, 16)
        g = torch.Generator().manual_seed(5)
        shape = paged.cache.v_scale.shape
        s = torch.ldexp(paged.cache.v_scale.cpu().nan_to_num(1.0), torch.randint(-30, 10, shape, generator=g))
        s[torch.rand(shape, generator=g) < 0.2] = 0
        paged.cache.v_scale.copy_(s)
        paged.cache.v[(s == 0).to(DEV).repeat_interleave(BLOCK, -1)] = 0
        q = _randn(sum(news), 8, 128) * 2
        cu = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device=DEV)
        out, lse = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, cu)
        _check_attention(paged, q, out, lse, news, True, 128 ** -0.5, rows=9)


def test_attention_a_nan_query_stays_in_its_row():
    for lens, news in (([50, 90], [1, 1]), ([200, 90], [150, 64])):
        paged, q, out, lse, cu = _attend(lens, news, 8, 2, 128, 16, rows=3)
        bad = q.clone()
        bad[news[0], 3, 7] = float("nan")
        bad[0, 1, 0] = float("inf")
        out2, lse2 = cr.attn_kv8(bad, paged.cache, paged.table_dev, paged.kv_len, cu)
        hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
        hit[news[0], 3] = hit[0, 1] = True
        assert out2[hit].isnan().all()
        assert torch.equal(out2[~hit], out[~hit]) and torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("lens,news,hidden", [([98], [4], 2), ([200], [200], 160), ([4000], [24], 8), ([1000], [517], 29)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_attention_rows_do_not_feel_what_they_do_not_see(lens, news, hidden, which, value):
    """A later block whose scale is not finite: the `hidden` rows in front of it give what they gave."""
    paged = Paged(lens, 1, 128, 16)
    q = _randn(news[0], 8, 128)
    cu = torch.tensor([0, news[0]], dtype=torch.int32, device=DEV)
    out, lse = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, cu)
    first = lens[0] - news[0] + hidden                       # the block's first token
    assert first % BLOCK == 0
    scales = paged.cache.k_scale if which == "k" else paged.cache.v_scale
    scales[int(paged.table[0, first // 16]), 0, 0] = value
    out2, lse2 = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, cu)
    assert torch.equal(out2[:hidden], out[:hidden]) and torch.equal(lse2[:hidden], lse[:hidden])


@pytest.mark.parametrize("lens,news", [([5], [1]), ([70], [3]), ([200], [200]), ([3000], [24])])
def test_attention_an_infinite_query_never_counts_as_unseen(lens, news):
    """A query whose scores are all -infinity (no codes of the other sign or zero in its way) is no row that sees nothing."""
    paged = Paged(lens, 1, 128, 16)
    paged.cache.k[..., 7] = 50
    q = _randn(news[0], 8, 128)
    cu = torch.tensor([0, news[0]], dtype=torch.int32, device=DEV)
    out, lse = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, cu)
    bad = q.clone()
    bad[0, 1, 7] = float("-inf")
    bad[-1, 6, 7] = float("-inf")
    out2, lse2 = cr.attn_kv8(bad, paged.cache, paged.table_dev, paged.kv_len, cu)
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
    hit[0, 1] = hit[-1, 6] = True
    assert out2[hit].isnan().all() and lse2[hit].isnan().all()
    assert torch.equal(out2[~hit], out[~hit]) and torch.equal(lse2[~hit], lse[~hit])


def test_attention_strided_queries_and_rows_behind():
    hq, hk, dim = 8, 2, 128
    paged = Paged([150, 33], hk, dim, 32)
    for news, total in (([1, 1], None), ([140, 33], 180), ([5, 2], 9)):
        rows = total or 2
        qkv = _randn(rows, hq + 2 * hk, dim)
        q = qkv[:, :hq]
        cu = None if total is None else torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device=DEV)
        out = torch.full((rows, hq, dim), 3.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((rows, hq), 3.0, device=DEV)
        cr.AttnKV8(q, paged.cache, paged.table_dev, paged.kv_len, out, cu=cu, lse=lse)()
        ref, _ = cr.attn_kv8(q.contiguous(), paged.cache, paged.table_dev, paged.kv_len, cu)
        n = sum(news)
        assert torch.equal(out[:n], ref[:n]) and (out[n:] == 3).all() and (lse[n:] == 3).all()
        _check_attention(paged, q, out, lse, news, True, dim ** -0.5, rows=9)
        # head-major queries
        qt = q.transpose(0, 1).contiguous().transpose(0, 1)
        out2, _ = cr.attn_kv8(qt, paged.cache, paged.table_dev, paged.kv_len, cu)
        assert torch.equal(out2[:n], ref[:n])


def test_attention_bad_device_arguments_are_recorded():
    hq, hk, dim = 4, 2, 64
    for lens, news in (([100, 60], [1, 1]), ([100, 60], [90, 60])):
        paged = Paged(lens, hk, dim, 16)
        q = _randn(sum(news), hq, dim)
        cu = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device=DEV)
        good, _ = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, cu)
        cr.convrot_device_status()
        table = paged.table_dev.clone()
        table[0, 2] = paged.cache.k.shape[0]
        table[0, 3] = -7
        out, _ = cr.attn_kv8(q, paged.cache, table, paged.kv_len, cu)
        assert torch.equal(out[news[0]:], good[news[0]:]) and out.isfinite().all()
        with pytest.raises(cr.ConvrotError):
            cr.convrot_device_status()
        for kv in ([10 ** 6, 60], [-5, 60]):
            out, _ = cr.attn_kv8(q, paged.cache, paged.table_dev, torch.tensor(kv, dtype=torch.int32, device=DEV), cu)
            assert torch.equal(out[news[0]:], good[news[0]:])
            with pytest.raises(cr.ConvrotError):
                cr.convrot_device_status()
        for bad in ([3, sum(news), sum(news)], [0, 10 ** 6, 10 ** 6], [0, sum(news), sum(news) - 1], [-4, 1, sum(news)]):
            cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, torch.tensor(bad, dtype=torch.int32, device=DEV))
            with pytest.raises(cr.ConvrotError):
                cr.convrot_device_status()


@pytest.mark.parametrize("cu", [[0, 12000, 13000, 14000, 0, 0], [0, 12000, 13000, 14000, -2000, 0], [0, 9000, 200, 13000, 100, 14000],
                                [13000, 0, 14000, 5, 14000, 6]])
def test_a_decreasing_cu_stays_in_bounds(cu):
    """Out of contract, recorded, and nothing beside the rows of the call and the sequences' own tokens is written."""
    batch, tokens, hq, hk, dim, page = 5, 14000, 8, 1, 64, 64
    wide = 16
    paged = Paged([wide * page] * batch, hk, dim, page, spare=6)
    cache = paged.cache
    table = paged.table_dev[:, :wide].contiguous()
    used = torch.zeros(cache.k.shape[0], dtype=torch.bool, device=DEV)
    used[table.flatten().long()] = True
    cu, kv = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu, [1000] * batch))
    k, v = _randn(tokens, hk, dim), _randn(tokens, hk, dim, seed=1)
    before = [x[~used].clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    cr.kv8_append(None, k, v, cache, table, kv, cu)
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()
    for x, y in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
        assert torch.equal(x.nan_to_num(7), y[~used].nan_to_num(7))
    room = torch.full((tokens + 8192, hq, dim), 5.0, dtype=torch.bfloat16, device=DEV)
    out, lse = room[4096:4096 + tokens], torch.zeros(tokens, hq, device=DEV)
    cr.AttnKV8(_randn(tokens, hq, dim), cache, table, kv, out, cu=cu, lse=lse)()
    assert (room[:4096] == 5).all() and (room[4096 + tokens:] == 5).all()
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()
    read = torch.full((tokens + 8192, hk, dim), 5.0, dtype=torch.bfloat16, device=DEV)
    cr.KV8Read(cache, table, kv, read[4096:4096 + tokens], None, cu=cu)()
    assert (read[:4096] == 5).all() and (read[4096 + tokens:] == 5).all()
    cr.load_library().convrot_device_status(None)


@pytest.mark.parametrize("cu", [[0, 60, 200], [-4, 60, 130], [3, 60, 130], [0, 130, 131], [-9, 0, 130]])
def test_read_records_rows_that_are_no_partition(cu):
    paged = Paged([100, 130], 2, 64, 16)
    out = torch.zeros(130, 2, 64, dtype=torch.bfloat16, device=DEV)
    cr.KV8Read(paged.cache, paged.table_dev, paged.kv_len, out, None, cu=torch.tensor(cu, dtype=torch.int32, device=DEV))()
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()


def test_attention_records_a_bad_cu_that_leaves_no_rows():
    paged = Paged([100], 1, 64, 16)
    for tokens in (1, 700):
        q = _randn(tokens, 8, 64)
        cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, torch.tensor([0, -5], dtype=torch.int32, device=DEV))
        with pytest.raises(cr.ConvrotError):
            cr.convrot_device_status()


@pytest.mark.parametrize("cu", [[0, 60, 200], [-4, 60, 130], [3, 60, 130], [0, 130, 131], [-9, 0, 130], [0, 130, 60]])
def test_append_and_attention_record_rows_that_are_no_partition(cu):
    paged = Paged([200, 200], 1, 64, 16)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    k, q = _randn(130, 1, 64), _randn(130, 4, 64)
    cr.kv8_append(q, k, k, paged.cache, paged.table_dev, paged.kv_len, cu)
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()
    cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, cu)
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()


def test_a_length_beyond_the_table_is_recorded_by_every_call():
    paged = Paged([100, 40], 2, 64, 16)
    q, k = _randn(2, 8, 64), _randn(2, 2, 64)
    kv = torch.tensor([2 ** 31 - 1, 40], dtype=torch.int32, device=DEV)
    good, _ = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len)
    for call in (lambda: cr.attn_kv8(q, paged.cache, paged.table_dev, kv), lambda: cr.kv8_read(paged.cache, paged.table_dev, kv),
                 lambda: cr.kv8_append(q, k, k, paged.cache, paged.table_dev, kv)):
        got = call()
        with pytest.raises(cr.ConvrotError):
            cr.convrot_device_status()
        assert got[0].isfinite().all()
    out, _ = cr.attn_kv8(q, paged.cache, paged.table_dev, kv)
    assert torch.equal(out[1:], cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len)[0][1:]) and good.isfinite().all()
    with pytest.raises(cr.ConvrotError):
        cr.convrot_device_status()


def test_attention_bits_do_not_change_between_runs_and_the_workspace_is_reused():
    lens, news = [3000, 10, 700], [1, 1, 1]
    paged = Paged(lens, 2, 128, 64)
    q = _randn(3, 16, 128)
    out, lse = torch.empty_like(q), torch.empty(3, 16, device=DEV)
    call = cr.AttnKV8(q, paged.cache, paged.table_dev, paged.kv_len, out, lse=lse)
    call()
    first = out.clone(), lse.clone()
    for _ in range(20):
        out.zero_()
        call()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    # other lengths on the same workspace
    paged.kv_len.copy_(torch.tensor([17, 9, 650]))
    paged.lens = [17, 9, 650]
    call()
    _check_attention(paged, q, out, lse, news, True, 128 ** -0.5)


def test_attention_one_workspace_for_calls_of_all_shapes():
    """Tiles of 8 and of 16 rows, many of them cut, and prompts with shared passes, one after another on one workspace of
    the largest size: each gives what it gives on its own."""
    hq, hk, dim = 16, 2, 128
    paged = Paged([9000, 7000], hk, dim, 64)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)        # noqa: E731
    jobs = {}
    for name, lens, news, cu in (("pairs", [9000, 7000], [2, 2], ints(0, 2, 4)), ("single", [9000, 7000], [1, 1], None),
                                 ("chunk", [9000], [24], ints(0, 24)), ("mixed", [9000, 3000], [40, 1], ints(0, 40, 41))):
        q = _randn(sum(news), hq, dim, seed=len(jobs)) * 2
        kv = ints(*lens)
        table = paged.table_dev[:len(lens)]
        own = cr.attn_kv8(q, paged.cache, table, kv, cu)
        paged.lens = lens
        _check_attention(paged, q, *own, news, True, dim ** -0.5, rows=3)
        out, lse = torch.empty_like(own[0]), torch.empty_like(own[1])
        jobs[name] = own, out, lse, (q, paged.cache, table, kv, out), dict(cu=cu, lse=lse)
    size = max(cr.AttnKV8(*j[3], **j[4]).ws_bytes for j in jobs.values())
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    calls = {name: cr.AttnKV8(*j[3], **j[4], ws=ws) for name, j in jobs.items()}
    order = ["pairs", "single", "pairs", "chunk", "single", "mixed", "single", "chunk", "pairs", "mixed", "pairs", "single"]
    for name in order:
        own, out, lse = jobs[name][:3]
        out.zero_()
        lse.zero_()
        calls[name]()
        assert torch.equal(out, own[0]) and torch.equal(lse, own[1]), name
    # and as captured steps that are replayed in turn
    graphs = {}
    for name in jobs:
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            calls[name]()
    for name in order:
        own, out, lse = jobs[name][:3]
        out.zero_()
        lse.zero_()
        graphs[name].replay()
        assert torch.equal(out, own[0]) and torch.equal(lse, own[1]), name
    cr.convrot_device_status()


@pytest.mark.parametrize("news", [[1, 1, 1], [200, 1, 30]])
def test_a_captured_step_follows_its_tensors(news):
    """Append and attention in one CUDA graph: replays take new lengths and values from the same tensors."""
    hq, hk, dim, page = 8, 2, 128, 16
    lens = [230, 40, 100]
    paged = _roomy(lens, [600, 600, 600], hk, dim, page)
    total = sum(news)
    qkv = _randn(total, hq + 2 * hk, dim)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    rot, out, lse = torch.empty(total, hq, dim, dtype=torch.bfloat16, device=DEV), None, torch.empty(total, hq, device=DEV)
    out = torch.empty_like(rot)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV)
    rope = cr.Rope(cr.rope_table(600, dim))
    append = cr.KV8Append(q, k, v, paged.cache, paged.table_dev, paged.kv_len, rot, cu=cu, rope=rope)
    attn = cr.AttnKV8(rot, paged.cache, paged.table_dev, paged.kv_len, out, cu=cu, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        append()
        attn()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append()
        attn()
    for step in range(1, 4):
        lens = [n + 7 * step for n in lens]
        paged.kv_len.copy_(torch.tensor(lens))
        # lengths jump by more than the rows: the tokens between hold random codes, give their blocks scales
        for s in (paged.cache.k_scale, paged.cache.v_scale):
            s.nan_to_num_(nan=0.01)
        paged.lens = lens
        qkv.copy_(_randn(total, hq + 2 * hk, dim, seed=step))
        graph.replay()
        torch.cuda.synchronize()
        _check_attention(paged, rot, out, lse, news, True, dim ** -0.5, rows=4)
    cr.convrot_device_status()


def test_the_first_call_of_a_process_may_be_captured():
    import subprocess
    import sys
    code = """
import torch
import rotated_int8_quantized_b200 as cr
q = torch.randn(200, 8, 64, device="cuda").bfloat16()
cache = cr.make_kv8_cache(20, 2, 64, 16)
table = torch.arange(20, dtype=torch.int32, device="cuda").view(1, 20)
kv = torch.tensor([200], dtype=torch.int32, device="cuda")
cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
k = torch.randn(200, 2, 64, device="cuda").bfloat16()
out, rot = torch.empty_like(q), torch.empty_like(q)
append = cr.KV8Append(q, k, k, cache, table, kv, rot, cu=cu, rope=cr.Rope(cr.rope_table(300, 64)))
attn = cr.AttnKV8(rot, cache, table, kv, out, cu=cu)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    append()
    attn()
g.replay()
torch.cuda.synchronize()
got = out.clone()
append()
attn()
assert torch.equal(got, out) and out.abs().max() > 0
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=__import__("os").path.dirname(__import__("os").path.dirname(__import__("os").path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_two_streams_at_once():
    """Calls with workspaces of their own, running at the same time."""
    jobs = []
    for i, (lens, news) in enumerate((([5000, 3], [1, 1]), ([600, 350], [600, 50]), ([4000], [1]), ([900], [900]))):
        paged = Paged(lens, 2, 128, 64, seed=i)
        q = _randn(sum(news), 8, 128, seed=i)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV)
        call = cr.AttnKV8(q, paged.cache, paged.table_dev, paged.kv_len, out, cu=cu, lse=lse)
        call()
        torch.cuda.synchronize()
        jobs.append((call, out, lse, out.clone(), lse.clone(), torch.cuda.Stream()))
    for _ in range(10):
        for call, out, _, _, _, stream in jobs:
            call(stream)
    torch.cuda.synchronize()
    for _, out, lse, ref, ref_lse, _ in jobs:
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_a_first_call_on_another_stream_finds_its_workspace_cleared():
    """The workspace that AttnKV8 makes is cleared on the stream of its construction, here far behind."""
    paged = Paged([9000, 7000], 2, 128, 64)
    q = _randn(2, 16, 128)
    want, want_lse = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len)
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    size = cr.AttnKV8(q, paged.cache, paged.table_dev, paged.kv_len, out, lse=lse).ws_bytes
    side = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        lse.zero_()
        used = torch.full((size,), 0x3F, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)                       # about a tenth of a second
        del used
        call = cr.AttnKV8(q, paged.cache, paged.table_dev, paged.kv_len, out, lse=lse)
        call(side)
        call(side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # made on a side stream, first called on the default one; and one that is first called in a capture
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        call = cr.AttnKV8(q, paged.cache, paged.table_dev, paged.kv_len, out, lse=lse)
    out.zero_()
    call()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    call = cr.AttnKV8(q, paged.cache, paged.table_dev, paged.kv_len, out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        inside, _ = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len)
    for _ in range(2):
        out.zero_()
        inside.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(inside, want)
        out.zero_()
        torch.cuda.synchronize()
        call(side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("as_handle", [False, True])
def test_functions_on_another_stream(as_handle):
    """stream= given as a stream or as its handle, the current stream far behind: what they make is made there."""
    hq, hk, dim, news = 8, 2, 64, [50, 1, 3]
    lens = [90, 700, 3]
    paged = _roomy([a - b for a, b in zip(lens, news)], lens, hk, dim, 16)
    paged.kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 50, 51, 54], dtype=torch.int32, device=DEV)
    qkv, w, rope = _randn(54, hq + 2 * hk, dim), _randn(dim, seed=1), cr.Rope(cr.rope_table(700, dim))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    pos = torch.arange(54, dtype=torch.int32, device=DEV)

    def step(**on):
        a, b = cr.qk_norm_rope(q, k, w, w, rope=rope, positions=pos, **on)
        r = cr.kv8_append(q, k, v, paged.cache, paged.table_dev, paged.kv_len, cu, w, w, rope=rope, **on)
        return [a, b, r, *cr.attn_kv8(r, paged.cache, paged.table_dev, paged.kv_len, cu, **on),
                *cr.kv8_read(paged.cache, paged.table_dev, paged.kv_len, 54, cu, **on)]

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        got = step(stream=side.cuda_stream if as_handle else side)
        side.synchronize()
        with torch.cuda.stream(side):
            assert all(torch.equal(x, y) for x, y in zip(got, want))
        del got
    cr.convrot_device_status()


def test_offsets_beyond_32_bits():
    """Codes of the last pages lie more than 2^32 bytes into the cache."""
    hk, dim, page = 8, 128, 128
    pages = 2 ** 32 // (hk * page * dim) + 40
    cache = cr.make_kv8_cache(pages, hk, dim, page)
    table = torch.tensor([[pages - 1, 0, pages - 3], [pages - 5, pages - 2, 1]], dtype=torch.int32, device=DEV)
    news = [300, 200]
    k, v = _randn(500, hk, dim), _randn(500, hk, dim, seed=1)
    cu = torch.tensor([0, 300, 500], dtype=torch.int32, device=DEV)
    kv = torch.tensor(news, dtype=torch.int32, device=DEV)
    cr.kv8_append(None, k, v, cache, table, kv, cu)
    kb, vb = cr.kv8_read(cache, table, kv, 500, cu)
    # within half a step of a block's scale, which is at most its largest value / 127, and the BF16 rounding
    for x, y in ((k, kb), (v, vb)):
        assert ((x.float() - y.float()).abs() <= x.float().abs().max() * (0.51 / 127 + 2.0 ** -8)).all()
    small = Paged(news, hk, dim, page)
    small.table = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32)
    at = table.long()
    small.cache = cr.KV8Cache(*(x[at.flatten()].contiguous() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    for rows in ([1, 1], [300, 200]):
        q = _randn(sum(rows), 16, dim)
        cu = torch.tensor([0, rows[0], sum(rows)], dtype=torch.int32, device=DEV)
        out, lse = cr.attn_kv8(q, cache, table, kv, cu)
        small.lens = news
        _check_attention(small, q, out, lse, rows, True, dim ** -0.5, rows=3)


def test_the_most_heads_and_eight_axes():
    heads, dim = 4096, 64
    x, w = _randn(3, heads, dim), _randn(dim, seed=1)
    table = cr.rope_table(100, dim, 1e4)
    pos = torch.randint(0, 100, (8, 3), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    axis = (torch.arange(dim // 2) % 8).to(torch.uint8)
    rope = cr.Rope(table, False, axis.to(DEV))
    ref = norm_rotate(bits_to_f64(x), bits_to_f64(w), 1e-6, table.cpu().numpy().astype(np.float64), pos.numpy(), axis.numpy(), False)
    for y in cr.qk_norm_rope(x, x, w, w, rope=rope, positions=pos.to(DEV)):
        _near_bf16(y, ref, np.abs(ref).max(-1, keepdims=True))
    paged = _roomy([0], [3], heads, dim, 16)
    q, k, v, _, old, before = _append(paged, [3], 0, heads, dim, 5)
    _check_append(paged, [3], bits_to_f64(k), bits_to_f64(v), old, before)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    out, lse = cr.attn_kv8(x, paged.cache, paged.table_dev, paged.kv_len, cu)
    _check_attention(paged, x, out, lse, [3], True, dim ** -0.5, rows=1)
    # one key head for all of them: 4096 rows a token
    _attend([37, 5], [2, 1], heads, 1, dim, 16, rows=1)
    _attend([37], [1], heads, 1, dim, 16, cu=False)
    cr.convrot_device_status()


def test_shared_pages_and_a_sequence_taken_back():
    """Two sequences with the same full pages in front, each with pages of its own behind; then one is taken back by some
    tokens and appended to again."""
    hk, dim, page = 2, 64, 32
    paged = Paged([64 + 9, 64 + 30], hk, dim, page)
    paged.table[1, :2] = paged.table[0, :2]
    paged.table_dev = paged.table.to(DEV)
    q, k, v, _, old, before = _append(paged, [5, 2], 0, hk, dim, 1)
    _check_append(paged, [5, 2], bits_to_f64(k), bits_to_f64(v), old, before)
    for news in ([1, 1], [60, 1]):
        x = _randn(sum(news), 8, dim)
        cu = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device=DEV)
        out, lse = cr.attn_kv8(x, paged.cache, paged.table_dev, paged.kv_len, cu)
        _check_attention(paged, x, out, lse, news, True, dim ** -0.5, rows=5)
    paged.lens = [64 + 9 + 5 - 3, 64 + 32]
    q, k, v, _, old, before = _append(paged, [8, 0], 0, hk, dim, 2)
    _check_append(paged, [8, 0], bits_to_f64(k), bits_to_f64(v), old, before)
    cr.convrot_device_status()


def test_outputs_that_are_not_asked_for():
    paged = Paged([100, 40], 2, 64, 16)
    cu = torch.tensor([0, 90, 95], dtype=torch.int32, device=DEV)
    k, v = cr.kv8_read(paged.cache, paged.table_dev, paged.kv_len, 95, cu)
    for which, want in ((0, k), (1, v)):
        got = torch.zeros_like(want)
        cr.KV8Read(paged.cache, paged.table_dev, paged.kv_len, got if which == 0 else None, got if which else None, cu=cu)()
        assert torch.equal(got, want)
    q = _randn(95, 8, 64)
    want, _ = cr.attn_kv8(q, paged.cache, paged.table_dev, paged.kv_len, cu)
    out = torch.zeros_like(q)
    cr.AttnKV8(q, paged.cache, paged.table_dev, paged.kv_len, out, cu=cu)()
    assert torch.equal(out, want)


def test_a_layer_from_projections_to_output():
    """INT8 q/k/v projections, append, attention, INT8 output projection: prompt in two chunks, then single tokens, against
    the same operators in 64 bits on the values the projections gave."""
    hq, hk, dim, hidden = 8, 2, 64, 256
    ws = [(_randn(n * dim, hidden, seed=n).float() * 0.05).bfloat16() for n in (hq, hk, hk)] + \
         [(_randn(hidden, hq * dim, seed=77).float() * 0.05).bfloat16()]
    wq = [cr.quantize_weight(w) for w in ws]
    nq, nk = _randn(dim, seed=5), _randn(dim, seed=6)
    table, eps = cr.rope_table(200, dim), 1e-6
    cs = table.cpu().numpy().astype(np.float64)
    steps = [[50, 20], [33, 7], [1, 1], [1, 1], [1, 1]]
    paged = _roomy([0, 0], [100, 40], hk, dim, 16)
    for i, news in enumerate(steps):
        total = sum(news)
        x = _randn(total, hidden, seed=i)
        qkv = [torch.empty(total, w.n, dtype=torch.bfloat16, device=DEV) for w in wq[:3]]
        cr.LinearBatch([x] * 3, wq[:3], qkv)()
        q, k, v = (y.view(total, -1, dim) for y in qkv)
        old = list(paged.lens)
        paged.lens = [a + b for a, b in zip(old, news)]
        paged.kv_len = torch.tensor(paged.lens, dtype=torch.int32, device=DEV)
        cu = torch.tensor([0, news[0], total], dtype=torch.int32, device=DEV)
        rot = cr.kv8_append(q, k, v, paged.cache, paged.table_dev, paged.kv_len, cu, nq, nk, eps, cr.Rope(table))
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(old, news)])[None]
        ref = norm_rotate(bits_to_f64(q), bits_to_f64(nq), eps, cs, pos, None, False)
        _near_bf16(rot, ref, np.abs(ref).max(-1, keepdims=True))
        out, lse = cr.attn_kv8(rot, paged.cache, paged.table_dev, paged.kv_len, cu)
        _check_attention(paged, rot, out, lse, news, True, dim ** -0.5, rows=5)
        y = cr.linear_int8(out.view(total, -1), wq[3], cr.make_workspace(total, wq[3]))
        assert y.isfinite().all()
    cr.convrot_device_status()
