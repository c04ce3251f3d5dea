"""CPU tests of the linear, gated and gradient clipping ABIs' host half
(include/linear.h, include/grad_clip.h; no GPU is touched): the ctypes mirrors
match the headers, every refusal returns its status before anything is enqueued,
overlaps of strided operands are told apart, scratch figures are shape-only."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest

import convolution_forward_amd as cf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40  # never dereferenced: the checks do range arithmetic only
GB = 1 << 32


@pytest.mark.parametrize("header,struct", [
    ("linear.h", "linear_problem"), ("linear.h", "gated_problem"), ("grad_clip.h", "grad_tensor"),
    ("grad_clip.h", "grad_clip_problem")])
def test_struct_layout_matches_header(header, struct):
    src = open(os.path.join(ROOT, "include", header)).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = []
    for decl in body.split(";"):
        decl = decl.strip()
        if decl:
            ctype, names = re.match(r"((?:const )?\w+\*?)\s+(.*)", decl, re.S).groups()
            fields += [(nm.strip(), ctype) for nm in names.split(",")]
    mirror = getattr(cf, struct)._fields_
    assert [f[0] for f in fields] == [m[0] for m in mirror]
    sizes = {"int64_t": 8, "int32_t": 4, "float": 4}
    for (name, ct), (_, mt) in zip(fields, mirror):
        assert (8 if ct.endswith("*") else sizes[ct]) == ctypes.sizeof(mt), name


def at(i):
    return FAKE + i * GB


def linear(p, dtype="f16", **kw):
    a = dict(x=at(0), w=at(1), b=at(2), r=at(3), y=at(4), z=at(5), scratch=at(9),
             scratch_bytes=1 << 30)
    a.update(kw)
    return cf.linear_check(p, dtype, **a)


def linear_back(p, dtype="f16", **kw):
    a = dict(x=at(0), w=at(1), z=at(2), dy=at(3), dx=at(4), dw=at(5), db=at(6), dr=None,
             scratch=at(9), scratch_bytes=1 << 30)
    a.update(kw)
    return cf.linear_backward_check(p, dtype, **a)


def gated(p, dtype="f16", **kw):
    a = dict(x=at(0), wg=at(1), wu=at(2), bg=at(3), bu=at(4), h=at(5), pg=at(6), pu=at(7),
             scratch=at(9), scratch_bytes=1 << 30)
    a.update(kw)
    return cf.gated_check(p, dtype, **a)


def gated_back(p, dtype="f16", **kw):
    a = dict(x=at(0), wg=at(1), wu=at(2), pg=at(3), pu=at(4), dh=at(5), dx=at(6), dwg=at(7),
             dwu=at(8), dbg=at(10), dbu=at(11), scratch=at(9), scratch_bytes=1 << 30)
    a.update(kw)
    return cf.gated_backward_check(p, dtype, **a)


def test_good_calls_pass():
    for dt in ("f32", "f16", "bf16"):
        assert linear(cf.make_linear_problem(4, 8, 16, bias=True, residual="before", save_z=True),
                      dt) == cf.CONV_OK
        assert linear_back(cf.make_linear_problem(4, 8, 16, act="gelu"), dt) == cf.CONV_OK
        assert gated(cf.make_gated_problem(4, 8, 16, bias=True, save=True), dt) == cf.CONV_OK
        assert gated_back(cf.make_gated_problem(4, 8, 16), dt) == cf.CONV_OK


@pytest.mark.parametrize("field,value,status", [
    ("m", -1, cf.CONV_ERR_SHAPE), ("m", 1 << 31, cf.CONV_ERR_SHAPE), ("n", 0, cf.CONV_ERR_SHAPE),
    ("k", 0, cf.CONV_ERR_SHAPE), ("n", (1 << 20) + 1, cf.CONV_ERR_SHAPE),
    ("k", (1 << 20) + 1, cf.CONV_ERR_SHAPE), ("ldx", 15, cf.CONV_ERR_SHAPE),
    ("ldw", (1 << 20) + 1, cf.CONV_ERR_SHAPE), ("ldy", 7, cf.CONV_ERR_SHAPE),
    ("ldr", -1, cf.CONV_ERR_SHAPE), ("ldz", 1, cf.CONV_ERR_SHAPE), ("lddx", 3, cf.CONV_ERR_SHAPE),
    ("lddw", 3, cf.CONV_ERR_SHAPE), ("lddr", 3, cf.CONV_ERR_SHAPE),
    ("x_off", -1, cf.CONV_ERR_ARG), ("dw_off", -1, cf.CONV_ERR_ARG),
    ("x_off", (1 << 62), cf.CONV_ERR_SHAPE), ("db_off", (1 << 62), cf.CONV_ERR_SHAPE),
    ("activation", 11, cf.CONV_ERR_ARG), ("activation", -1, cf.CONV_ERR_ARG),
    ("has_bias", 2, cf.CONV_ERR_ARG), ("has_residual", 3, cf.CONV_ERR_ARG),
    ("save_z", 2, cf.CONV_ERR_ARG), ("w_layout", 2, cf.CONV_ERR_ARG),
    ("reserved", 1, cf.CONV_ERR_ARG)])
def test_linear_refusals(field, value, status):
    p = cf.make_linear_problem(4, 8, 16, bias=True)
    setattr(p, field, value)
    assert linear(p) == status
    assert linear_back(p) == status
    n = ctypes.c_uint64()
    assert cf.lib().linear_scratch_size(ctypes.byref(p), 1, ctypes.byref(n)) == status
    assert cf.lib().linear_backward_scratch_size(ctypes.byref(p), 1, ctypes.byref(n)) == status
    with pytest.raises(cf.ConvError):
        cf.linear_describe_variant(p, "f16")


@pytest.mark.parametrize("field,value,status", [
    ("m", -1, cf.CONV_ERR_SHAPE), ("f", 0, cf.CONV_ERR_SHAPE), ("k", 0, cf.CONV_ERR_SHAPE),
    ("f", (1 << 20) + 1, cf.CONV_ERR_SHAPE), ("ldx", 15, cf.CONV_ERR_SHAPE),
    ("ldw", 15, cf.CONV_ERR_SHAPE), ("ldh", 7, cf.CONV_ERR_SHAPE), ("ldp", 7, cf.CONV_ERR_SHAPE),
    ("lddx", 15, cf.CONV_ERR_SHAPE), ("lddw", 15, cf.CONV_ERR_SHAPE),
    ("wu_off", -1, cf.CONV_ERR_ARG), ("dbu_off", -1, cf.CONV_ERR_ARG),
    ("pu_off", (1 << 62), cf.CONV_ERR_SHAPE), ("activation", 11, cf.CONV_ERR_ARG),
    ("has_bias", -1, cf.CONV_ERR_ARG), ("save_p", 2, cf.CONV_ERR_ARG),
    ("reserved", 1, cf.CONV_ERR_ARG)])
def test_gated_refusals(field, value, status):
    p = cf.make_gated_problem(4, 8, 16)
    setattr(p, field, value)
    assert gated(p) == status
    assert gated_back(p) == status
    n = ctypes.c_uint64()
    assert cf.lib().gated_scratch_size(ctypes.byref(p), 1, ctypes.byref(n)) == status
    assert cf.lib().gated_backward_scratch_size(ctypes.byref(p), 1, ctypes.byref(n)) == status


def test_dtype_and_null_pointers():
    p = cf.make_linear_problem(4, 8, 16, bias=True, residual="after", save_z=True)
    for dt in (3, -1):
        assert linear(p, dt) == cf.CONV_ERR_ARG
        assert gated(cf.make_gated_problem(4, 8, 16), dt) == cf.CONV_ERR_ARG
    for name in ("x", "w", "b", "r", "y", "z"):
        assert linear(p, **{name: None}) == cf.CONV_ERR_ARG, name
    p = cf.make_linear_problem(4, 8, 16)  # nothing optional asked for
    assert linear(p, b=None, r=None, z=None) == cf.CONV_OK
    p = cf.make_linear_problem(4, 8, 16, act="silu")
    for name in ("x", "w", "z", "dy"):
        assert linear_back(p, **{name: None}) == cf.CONV_ERR_ARG, name
    assert linear_back(p, x=None, dw=None) == cf.CONV_OK
    assert linear_back(p, w=None, dx=None) == cf.CONV_OK
    assert linear_back(p, dx=None, dw=None, db=None) == cf.CONV_ERR_ARG  # nothing asked for
    assert linear_back(p, dr=at(7)) == cf.CONV_ERR_ARG  # no residual
    assert linear_back(cf.make_linear_problem(4, 8, 16), z=None) == cf.CONV_OK  # identity
    g = cf.make_gated_problem(4, 8, 16, bias=True, save=True)
    for name in ("x", "wg", "wu", "bg", "bu", "h", "pg", "pu"):
        assert gated(g, **{name: None}) == cf.CONV_ERR_ARG, name
    for name in ("x", "wg", "wu", "pg", "pu", "dh", "dwg", "dwu", "dbg", "dbu"):
        assert gated_back(g, **{name: None}) == cf.CONV_ERR_ARG, name
    assert gated_back(g, dx=None, wg=None, wu=None) == cf.CONV_OK
    assert gated_back(g, dwg=None, dwu=None, x=None) == cf.CONV_OK


def test_no_rows_need_no_row_operands():
    p = cf.make_linear_problem(0, 8, 16, residual="before", save_z=True)
    assert linear(p, x=None, r=None, y=None, z=None) == cf.CONV_OK
    assert linear_back(p, x=None, z=None, dy=None, dx=None) == cf.CONV_OK
    g = cf.make_gated_problem(0, 8, 16, save=True)
    assert gated(g, x=None, h=None, pg=None, pu=None) == cf.CONV_OK
    assert gated_back(g, x=None, pg=None, pu=None, dh=None, dx=None) == cf.CONV_OK


def test_misaligned_elements_and_scratch():
    p = cf.make_linear_problem(4, 8, 16)
    assert linear(p, x=at(0) + 1) == cf.CONV_ERR_ARG
    assert linear(p, "f32", y=at(4) + 2) == cf.CONV_ERR_ARG
    assert linear(p, "f16", y=at(4) + 2) == cf.CONV_OK
    p = cf.make_linear_problem(64, 64, 4096, w_layout="kn")  # few tiles, long k: split
    need = cf.linear_scratch_size(p, "f16")
    assert need > 0
    assert linear(p, scratch_bytes=need) == cf.CONV_OK
    assert linear(p, scratch_bytes=need - 256) == cf.CONV_ERR_SCRATCH
    assert linear(p, scratch=None) == cf.CONV_ERR_ARG
    assert linear(p, scratch=at(9) + 16) == cf.CONV_ERR_ARG
    assert linear(p, scratch=at(4)) == cf.CONV_ERR_OVERLAP
    assert linear(p, scratch=at(0)) == cf.CONV_ERR_OVERLAP


def test_overlap_rules():
    p = cf.make_linear_problem(4, 8, 16, residual="before", save_z=True)
    assert linear(p, y=at(3)) == cf.CONV_OK  # y = r exactly
    assert linear(p, y=at(3) + 16) == cf.CONV_ERR_OVERLAP
    assert linear(p, z=at(3)) == cf.CONV_ERR_OVERLAP
    assert linear(p, z=at(4)) == cf.CONV_ERR_OVERLAP
    assert linear(p, y=at(1)) == cf.CONV_ERR_OVERLAP
    assert linear(p, y=at(0) + 4 * 16 * 2) == cf.CONV_OK  # right behind x
    assert linear(p, y=at(0) + 4 * 16 * 2 - 2) == cf.CONV_ERR_OVERLAP
    # the halves of one [m, 2f] buffer, and halves that meet
    g = cf.make_gated_problem(4, 8, 16, save=True, ldp=16)
    assert gated(g, pg=at(6), pu=at(6) + 16) == cf.CONV_OK
    assert gated(g, pg=at(6) + 16, pu=at(6)) == cf.CONV_OK
    assert gated(g, pg=at(6), pu=at(6) + 14) == cf.CONV_ERR_OVERLAP
    assert gated(g, pg=at(6), pu=at(6) + 18) == cf.CONV_ERR_OVERLAP
    # dr over dy exactly, not partly
    p = cf.make_linear_problem(4, 8, 16, act="relu", residual="before")
    assert linear_back(p, dr=at(3)) == cf.CONV_OK
    assert linear_back(p, dr=at(3) + 2) == cf.CONV_ERR_OVERLAP
    assert linear_back(p, dw=at(1)) == cf.CONV_ERR_OVERLAP
    g = cf.make_gated_problem(4, 8, 16)
    assert gated_back(g, dwg=at(7), dwu=at(7)) == cf.CONV_ERR_OVERLAP
    assert gated_back(g, dx=at(5)) == cf.CONV_ERR_OVERLAP


def test_plans_are_named():
    name = lambda m, n, k, dt="bf16", **kw: cf.linear_describe_variant(  # noqa: E731
        cf.make_linear_problem(m, n, k, **kw), dt)
    assert name(1, 4096, 4096).startswith("linear.bf16.stream")
    assert name(8192, 4096, 4096) == "linear.bf16.tile256x256"
    assert cf.gated_describe_variant(cf.make_gated_problem(1, 512, 256), "f16").startswith(
        "gated.f16.stream")
    text = cf.linear_backward_describe_variant(cf.make_linear_problem(4096, 512, 512), "f32")
    assert re.match(r"linear_backward\.f32\.dx\.\S+\.dw\.\S+", text)
    assert cf.gated_backward_describe_variant(cf.make_gated_problem(64, 512, 512), "bf16")
    buf = ctypes.create_string_buffer(8)
    p = cf.make_linear_problem(4, 8, 16)
    assert cf.lib().linear_describe_variant(ctypes.byref(p), 1, buf, 8) == cf.CONV_ERR_ARG


def test_planners_reference_no_hip_symbol(tmp_path):
    if shutil.which("g++") is None or shutil.which("nm") is None:
        pytest.skip("no host toolchain")
    csrc = os.path.join(ROOT, "convolution_forward_amd", "csrc")
    for name in ("linear_plan.cpp", "grad_clip_plan.cpp"):
        obj = str(tmp_path / (name + ".o"))
        subprocess.check_call(["g++", "-std=c++17", "-c", "-I", os.path.join(ROOT, "include"), "-I",
                               csrc, os.path.join(csrc, name), "-o", obj])
        assert "hip" not in subprocess.check_output(["nm", "-u", "-C", obj], text=True).lower()


# ------------------------------------------------------------ gradient clipping

def clip(pairs, **kw):
    """pairs: (g, out, elems) by address."""
    return cf.make_grad_clip_problem([g for g, _, _ in pairs], [o for _, o, _ in pairs], "f32",
                                     elems=[e for _, _, e in pairs], **kw)


def clip_check(p, norm=at(20), scratch=at(21), scratch_bytes=1 << 30):
    return cf.grad_clip_check(p, norm, scratch, scratch_bytes)


def test_clip_refusals():
    good = [(at(0), at(1), 100), (at(2), at(2), 7), (0, 0, 0)]
    assert clip_check(clip(good)) == cf.CONV_OK
    assert clip_check(clip([])) == cf.CONV_OK
    for field, value in (("kind", 0), ("kind", 4), ("max_norm", -1.0), ("max_norm", math.nan),
                         ("eps", -1e-6), ("eps", math.nan), ("reserved", 1)):
        p = clip(good)
        setattr(p, field, value)
        assert clip_check(p) == cf.CONV_ERR_ARG, field
    for field, value, status in (("dtype", 3, cf.CONV_ERR_ARG), ("reserved", 1, cf.CONV_ERR_ARG),
                                 ("g", None, cf.CONV_ERR_ARG), ("out", None, cf.CONV_ERR_ARG),
                                 ("g", at(0) + 2, cf.CONV_ERR_ARG),
                                 ("elems", -1, cf.CONV_ERR_SHAPE),
                                 ("elems", 1 << 60, cf.CONV_ERR_SHAPE)):
        p = clip(good)
        setattr(p.tensors[0], field, value)
        assert clip_check(p) == status, field
    for count in (-1, 65537):
        p = clip(good)
        p.count = count
        assert clip_check(p) == cf.CONV_ERR_SHAPE
    assert clip_check(clip(good), norm=None) == cf.CONV_ERR_ARG
    assert clip_check(clip(good), norm=at(20) + 2) == cf.CONV_ERR_ARG
    assert clip_check(clip(good), scratch=None) == cf.CONV_ERR_ARG
    assert clip_check(clip(good), scratch=at(21) + 8) == cf.CONV_ERR_ARG
    need = cf.grad_clip_scratch_size(clip(good))
    assert clip_check(clip(good), scratch_bytes=need) == cf.CONV_OK
    assert clip_check(clip(good), scratch_bytes=need - 1) == cf.CONV_ERR_SCRATCH


def test_clip_overlaps():
    assert clip_check(clip([(at(0), at(0) + 4, 100)])) == cf.CONV_ERR_OVERLAP
    assert clip_check(clip([(at(0), at(0) + 400, 100)])) == cf.CONV_OK
    assert clip_check(clip([(at(0), at(1), 100)]), norm=at(0) + 396) == cf.CONV_ERR_OVERLAP
    assert clip_check(clip([(at(0), at(1), 100)]), scratch=at(1)) == cf.CONV_ERR_OVERLAP
    assert clip_check(clip([(at(0), at(1), 100)]), norm=at(21)) == cf.CONV_ERR_OVERLAP


def test_clip_norm_alone_and_scratch_by_lengths():
    p = cf.make_grad_clip_problem([at(0), at(1)], None, "f16", elems=[5, 0])
    assert clip_check(p) == cf.CONV_OK
    q = cf.make_grad_clip_problem([at(3), at(5)], None, "f32", elems=[5, 0])
    assert cf.grad_clip_scratch_size(p) == cf.grad_clip_scratch_size(q)
    with pytest.raises(KeyError):
        cf.make_grad_clip_problem([at(0)], None, "f16", elems=[5], norm=3)
