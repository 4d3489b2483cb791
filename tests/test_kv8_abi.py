"""The attention-side entry points without a GPU: argument checks on the
host, the binding's structs and its own checks."""
import ctypes
import os
import subprocess

import pytest
import torch

import rotated_int8_quantized_b200 as cr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, ALIGN, SHAPE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return cr.load_library()


def _cache(**kw):
    c = cr.convrot_kv8_t(0x10000, 0x20000, 0x30000, 0x40000, 8, 2, 64, 128)
    for name, v in kw.items():
        setattr(c, name, v)
    return c


def _seqs(**kw):
    s = cr.convrot_kv8_seqs_t(0x50000, 0x60000, 0x70000, 10, 2, 4)
    for name, v in kw.items():
        setattr(s, name, v)
    return s


def _rope(**kw):
    r = cr.convrot_rope_t(0x80000, 100, 128, 0, None, 1)
    for name, v in kw.items():
        setattr(r, name, v)
    return r


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(k=0), INVALID), (dict(v_scale=0), INVALID), (dict(pages=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(kv_heads=4097), SHAPE), (dict(page_tokens=8), SHAPE), (dict(page_tokens=48), SHAPE), (dict(page_tokens=2048), SHAPE),
    (dict(page_tokens=16), OK), (dict(page_tokens=1024), OK), (dict(head_dim=96), SHAPE), (dict(head_dim=64), OK),
    (dict(pages=2 ** 31), SHAPE), (dict(k=0x10008), ALIGN), (dict(k=0x10010), ALIGN),
    (dict(v=0x20010), ALIGN), (dict(k_scale=0x30004), ALIGN)])
def test_cache_handle(lib, kw, want):
    c, out = _cache(**kw), cr.convrot_kv8_t()
    assert lib.convrot_kv8_init(ctypes.byref(out), c.k, c.v, c.k_scale, c.v_scale, c.pages, c.kv_heads, c.page_tokens,
                                c.head_dim) == want
    assert out.pages == (c.pages if want == OK else 0)
    assert lib.convrot_kv8_init(None, c.k, c.v, c.k_scale, c.v_scale, 8, 2, 64, 128) == INVALID


def _norm_job(rope=None, **kw):
    j = cr.convrot_qk_norm_rope_t()
    j.tokens, j.q_heads, j.kv_heads, j.head_dim, j.eps = 10, 4, 2, 128, 1e-6
    for i, name in enumerate(("q", "k", "q_out", "k_out")):
        heads = 4 if name[0] == "q" else 2
        setattr(j, name, 0x100000 * (i + 1))
        setattr(j, name + "_token_stride", heads * 128)
        setattr(j, name + "_head_stride", 128)
    if rope is not None:
        j.rope, j.positions = ctypes.pointer(rope), 0x90000
    for name, v in kw.items():
        setattr(j, name, v)
    return j


# every call below is refused before a device is looked for
@pytest.mark.parametrize("kw,rope,want", [
    (dict(tokens=0), None, INVALID), (dict(q_heads=0), None, INVALID), (dict(kv_heads=-1), None, INVALID),
    (dict(head_dim=80), None, SHAPE), (dict(q_heads=5000), None, SHAPE), (dict(tokens=2 ** 30), None, SHAPE),
    (dict(q=0), None, INVALID), (dict(k=0), None, INVALID), (dict(q=0x100008), None, ALIGN),
    (dict(q_token_stride=516), None, ALIGN), (dict(k_head_stride=-128), None, INVALID),
    (dict(q_out_head_stride=64), None, INVALID), (dict(k_out_token_stride=128), None, INVALID),
    (dict(q_weight=0x8), None, ALIGN), (dict(eps=-1.0), None, INVALID), (dict(eps=float("nan")), None, INVALID),
    ({}, dict(cos_sin=0), INVALID), ({}, dict(rot_dim=12), SHAPE), ({}, dict(rot_dim=136), SHAPE), ({}, dict(rot_dim=0), SHAPE),
    ({}, dict(axes=9), INVALID), ({}, dict(axes=0), INVALID), ({}, dict(positions=0), INVALID), ({}, dict(cos_sin=0x80008), ALIGN),
    ({}, dict(axis=0x90002), ALIGN), (dict(positions=0), {}, INVALID), (dict(positions=0x90002), {}, ALIGN)])
def test_norm_rope_refusals(lib, kw, rope, want):
    job = _norm_job(None if rope is None else _rope(**rope), **kw)
    assert lib.convrot_qk_norm_rope(ctypes.byref(job), None) == want


SEQS = [(dict(page_table=0), INVALID), (dict(kv_len=0), INVALID), (dict(batch=0), INVALID), (dict(max_pages=0), INVALID),
        (dict(tokens=0), INVALID), (dict(cu=0), INVALID), (dict(cu=0x70002), ALIGN), (dict(tokens=2 ** 40), SHAPE),
        (dict(batch=2 ** 31 - 1), SHAPE)]


@pytest.mark.parametrize("kw,want", SEQS)
def test_sequence_refusals(lib, kw, want):
    c = _cache()
    read = cr.convrot_kv8_read_t(ctypes.pointer(c), _seqs(**kw), 0x100000, 0x200000)
    assert lib.convrot_kv8_read(ctypes.byref(read), None) == want
    append = _append_job(c, **kw)
    assert lib.convrot_kv8_append(ctypes.byref(append), None) == want
    attn = _attn_job(c, **kw)
    assert lib.convrot_attn_kv8(ctypes.byref(attn), 0x300000, 1 << 40, None) == want
    assert lib.convrot_attn_kv8_workspace_bytes(ctypes.byref(attn)) == 0


def _append_job(c, **seqs):
    j = cr.convrot_kv8_append_t()
    j.cache, j.seqs, j.q_heads, j.eps = ctypes.pointer(c), _seqs(**seqs), 4, 1e-6
    for i, name in enumerate(("q", "k", "v", "q_out")):
        heads = 4 if name[0] == "q" else 2
        setattr(j, name, 0x100000 * (i + 1))
        setattr(j, name + "_token_stride", heads * 128)
        setattr(j, name + "_head_stride", 128)
    return j


def _attn_job(c, **seqs):
    j = cr.convrot_attn_kv8_t()
    j.cache, j.seqs, j.q_heads, j.causal = ctypes.pointer(c), _seqs(**seqs), 4, 1
    j.q, j.q_token_stride, j.q_head_stride, j.out, j.lse, j.scale = 0x100000, 512, 128, 0x200000, 0x300000, 0.1
    return j


@pytest.mark.parametrize("kw,want", [
    (dict(q_heads=-1), INVALID), (dict(q_heads=4097), SHAPE), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(q=0), INVALID),
    (dict(q_out=0), INVALID), (dict(v_head_stride=4), ALIGN), (dict(q_out_token_stride=256), INVALID),
    (dict(k_weight=0x4), ALIGN), (dict(eps=float("inf")), INVALID)])
def test_append_refusals(lib, kw, want):
    j = _append_job(_cache())
    for name, v in kw.items():
        setattr(j, name, v)
    assert lib.convrot_kv8_append(ctypes.byref(j), None) == want
    assert lib.convrot_kv8_append(None, None) == INVALID


def test_append_without_positions_has_one_axis(lib):
    for kw in (dict(axes=2), dict(axis=0x90000)):
        j, r = _append_job(_cache()), _rope(**kw)
        j.rope = ctypes.pointer(r)
        assert lib.convrot_kv8_append(ctypes.byref(j), None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(q_heads=0), INVALID), (dict(q_heads=3), SHAPE), (dict(q_heads=4098), SHAPE), (dict(q=0), INVALID), (dict(out=0), INVALID),
    (dict(out=0x200008), ALIGN), (dict(lse=0x300002), ALIGN), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q_head_stride=100), ALIGN)])
def test_attention_refusals(lib, kw, want):
    j = _attn_job(_cache())
    for name, v in kw.items():
        setattr(j, name, v)
    assert lib.convrot_attn_kv8(ctypes.byref(j), 0x300000, 1 << 40, None) == want
    assert lib.convrot_attn_kv8_workspace_bytes(ctypes.byref(j)) == 0
    assert lib.convrot_attn_kv8(None, 0x300000, 1 << 40, None) == INVALID


def test_attention_workspace(lib):
    c = _cache()
    j = _attn_job(c)
    need = lib.convrot_attn_kv8_workspace_bytes(ctypes.byref(j))
    assert need > 0 and need % 256 == 0
    assert lib.convrot_attn_kv8(ctypes.byref(j), 0x300004, 1 << 40, None) == ALIGN
    if not torch.cuda.is_available():
        pytest.skip("the size is checked against a device's")
    assert lib.convrot_attn_kv8(ctypes.byref(j), None, 0, None) == 5
    assert lib.convrot_attn_kv8(ctypes.byref(j), 0x400000, need - 1, None) == 5


def test_bad_cache_in_a_job(lib):
    c = _cache(page_tokens=20)
    assert lib.convrot_attn_kv8(ctypes.byref(_attn_job(c)), 0x300000, 1 << 40, None) == SHAPE
    assert lib.convrot_kv8_append(ctypes.byref(_append_job(c)), None) == SHAPE
    read = cr.convrot_kv8_read_t(ctypes.pointer(_cache()), _seqs(), None, None)
    assert lib.convrot_kv8_read(ctypes.byref(read), None) == INVALID


def test_structs_match_the_header(tmp_path):
    names = ["convrot_kv8_t", "convrot_rope_t", "convrot_kv8_seqs_t", "convrot_qk_norm_rope_t", "convrot_kv8_append_t",
             "convrot_kv8_read_t", "convrot_attn_kv8_t"]
    lines = []
    for n in names:
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (n, n))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (n, f, n, f) for f, _ in getattr(cr, n)._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"convrot.h\"\nint main(void) {\n%s\nreturn 0;\n}\n"
                   % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = dict(line.split() for line in subprocess.check_output([str(exe)], text=True).splitlines())
    want = {}
    for n in names:
        t = getattr(cr, n)
        want[n] = ctypes.sizeof(t)
        want.update({"%s.%s" % (n, f): getattr(t, f).offset for f, _ in t._fields_})
    assert {k: int(v) for k, v in got.items()} == want


def test_rope_table_angles_are_taken_in_64_bits():
    t = cr.rope_table(70000, 64, 1e4, device="cpu")
    import math
    for p, i in ((0, 0), (1, 31), (69999, 0), (65537, 7)):
        a = p * 1e4 ** (-2 * i / 64)
        assert abs(t[p, i, 0].item() - math.cos(a)) <= 2 ** -24 and abs(t[p, i, 1].item() - math.sin(a)) <= 2 ** -24


def test_binding_refuses_wrong_tensors():
    with pytest.raises(ValueError):
        cr.KV8Cache(torch.zeros(2, 1, 16, 64, dtype=torch.int8), torch.zeros(2, 1, 16, 64, dtype=torch.int8),
                    torch.zeros(2, 1, 2), torch.zeros(2, 1, 1))
    with pytest.raises(ValueError):
        cr.KV8Cache(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 1), torch.zeros(2, 1, 1))
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                       # not on a GPU
        cr.QKNormRope(x, None, x, None)
    with pytest.raises(ValueError):
        cr.QKNormRope(x.float(), None, x, None)


def test_a_read_without_outputs_is_refused():
    class Cache:
        handle, k = _cache(), torch.zeros(1)
    with pytest.raises(ValueError):
        cr.KV8Read(Cache, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), None, None)
