"""CPU tests of the host half of layer norm, dropout, row quantization and the 8-bit
linear layer (no GPU is touched): the ctypes mirrors match the headers, every refusal
returns its status before anything is enqueued, overlaps of strided operands are told
apart, scratch is shape-only, the planners run clean under sanitizers; and the mask
reference of the GPU tests against the generator's published answers."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import convolution_forward_amd as cf
import mask_reference as mask

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_forward_amd", "csrc")
FAKE = 1 << 40  # never dereferenced: the checks do range arithmetic only
GB = 1 << 32
ARG, SHAPE, OVERLAP, SCRATCH = (cf.CONV_ERR_ARG, cf.CONV_ERR_SHAPE, cf.CONV_ERR_OVERLAP,
                                cf.CONV_ERR_SCRATCH)


@pytest.mark.parametrize("header,struct", [
    ("layer_norm.h", "layer_norm_problem"), ("dropout.h", "dropout_problem"),
    ("linear_int8.h", "quantize_problem"), ("linear_int8.h", "linear_int8_problem")])
def test_struct_layout_matches_header(header, struct):
    src = open(os.path.join(ROOT, "include", header)).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = []
    for decl in body.split(";"):
        if decl.strip():
            ctype, names = decl.strip().split(None, 1)
            fields += [(nm.strip(), ctype) for nm in names.split(",")]
    mirror = getattr(cf, struct)._fields_
    assert [f[0] for f in fields] == [m[0] for m in mirror]
    sizes = {"int64_t": 8, "uint64_t": 8, "int32_t": 4, "float": 4}
    for (name, ct), (_, mt) in zip(fields, mirror):
        assert sizes[ct] == ctypes.sizeof(mt), name


def at(i):
    return FAKE + i * GB


def norm(p, dtype="f16", **kw):
    a = dict(x=at(0), r=at(1), w=at(2), b=at(3), y=at(4), s=at(5), mean=at(6), rstd=at(7),
             step=at(8), scratch=at(9), scratch_bytes=1 << 30)
    a.update(kw)
    return cf.layer_norm_check(p, dtype, **a)


def norm_back(p, dtype="f16", **kw):
    a = dict(s=at(0), w=at(1), mean=at(2), rstd=at(3), dy=at(4), ds=at(5), dx=at(6), dr=at(7),
             dw=at(8), db=at(10), step=at(11), scratch=at(9), scratch_bytes=1 << 30)
    a.update(kw)
    return cf.layer_norm_backward_check(p, dtype, **a)


def drop(p, dtype="f16", **kw):
    a = dict(x=at(0), r=at(1), y=at(2), step=at(3))
    a.update(kw)
    return cf.dropout_check(p, dtype, **a)


def quant(p, dtype="f16", **kw):
    a = dict(x=at(0), q=at(1), scale=at(2))
    a.update(kw)
    return cf.quantize_check(p, dtype, **a)


def int8(p, dtype="f16", **kw):
    a = dict(x=at(0), xs=at(1), w=at(2), ws=at(3), b=at(4), r=at(5), y=at(6), scratch=at(9),
             scratch_bytes=1 << 30)
    a.update(kw)
    return cf.linear_int8_check(p, dtype, **a)


NORM = lambda **kw: cf.make_layer_norm_problem(4, 40, residual=True, drop=0.1, **kw)  # noqa: E731


def test_good_calls_pass():
    for dt in ("f32", "f16", "bf16"):
        assert norm(NORM(), dt) == norm_back(NORM(), dt) == cf.CONV_OK
        assert drop(cf.make_dropout_problem(4, 40, 0.5, residual=True), dt) == cf.CONV_OK
        assert quant(cf.make_quantize_problem(4, 40), dt) == cf.CONV_OK
        assert int8(cf.make_linear_int8_problem(4, 8, 40, bias=True, residual="before"), dt) == cf.CONV_OK
    p = cf.make_layer_norm_problem(4, 40, weight=False, bias=False)  # nothing optional asked for
    assert norm(p, r=None, w=None, b=None, s=None, mean=None, rstd=None, step=None) == cf.CONV_OK
    assert norm_back(p, w=None, ds=None, dr=None, dw=None, db=None, step=None) == cf.CONV_OK


@pytest.mark.parametrize("field,value,status", [
    ("m", -1, SHAPE), ("m", 1 << 31, SHAPE), ("n", 0, SHAPE), ("n", (1 << 20) + 1, SHAPE),
    ("ldx", 39, SHAPE), ("ldr", -1, SHAPE), ("ldy", 1, SHAPE), ("lds", (1 << 20) + 1, SHAPE),
    ("ldds", 39, SHAPE), ("lddx", 39, SHAPE), ("lddr", 39, SHAPE), ("x_off", -1, ARG),
    ("db_off", -1, ARG), ("s_off", 1 << 62, SHAPE), ("dw_off", 1 << 62, SHAPE),
    ("eps", -1e-6, ARG), ("eps", math.nan, ARG), ("eps", math.inf, ARG), ("drop", -0.1, ARG),
    ("drop", 1.01, ARG), ("drop", math.nan, ARG), ("has_weight", 2, ARG), ("has_bias", -1, ARG),
    ("has_residual", 2, ARG), ("reserved", 1, ARG)])
def test_layer_norm_refusals(field, value, status):
    p = NORM()
    setattr(p, field, value)
    assert norm(p) == status and norm_back(p) == status
    n = ctypes.c_uint64()
    assert cf.lib().layer_norm_scratch_size(ctypes.byref(p), 1, ctypes.byref(n)) == status
    assert cf.lib().layer_norm_backward_scratch_size(ctypes.byref(p), 1, ctypes.byref(n)) == status
    for describe in (cf.layer_norm_describe_variant, cf.layer_norm_backward_describe_variant):
        with pytest.raises(cf.ConvError):
            describe(p, "f16")


@pytest.mark.parametrize("field,value,status", [
    ("m", -1, SHAPE), ("m", 1 << 31, SHAPE), ("n", 0, SHAPE), ("n", (1 << 20) + 1, SHAPE),
    ("ldx", 39, SHAPE), ("ldr", 39, SHAPE), ("ldy", (1 << 20) + 1, SHAPE), ("x_off", -1, ARG),
    ("y_off", 1 << 62, SHAPE), ("drop", -0.1, ARG), ("drop", 1.5, ARG), ("drop", math.nan, ARG),
    ("has_residual", 2, ARG), ("reserved", 1, ARG)])
def test_dropout_refusals(field, value, status):
    p = cf.make_dropout_problem(4, 40, 0.5, residual=True)
    setattr(p, field, value)
    assert drop(p) == status
    assert cf.dropout_backward_check(p, "f16", at(0), at(1)) == status
    with pytest.raises(cf.ConvError):
        cf.dropout_describe_variant(p, "f16")


@pytest.mark.parametrize("field,value,status", [
    ("m", -1, SHAPE), ("n", 0, SHAPE), ("n", (1 << 20) + 1, SHAPE), ("ldx", 39, SHAPE),
    ("ldq", 39, SHAPE), ("q_off", -1, ARG), ("scale_off", 1 << 62, SHAPE), ("reserved", 1, ARG)])
def test_quantize_refusals(field, value, status):
    p = cf.make_quantize_problem(4, 40)
    setattr(p, field, value)
    assert quant(p) == status


@pytest.mark.parametrize("field,value,status", [
    ("m", -1, SHAPE), ("m", 1 << 31, SHAPE), ("n", 0, SHAPE), ("k", 0, SHAPE), ("k", 131072, SHAPE),
    ("n", (1 << 20) + 1, SHAPE), ("ldx", 39, SHAPE), ("ldw", 39, SHAPE), ("ldr", 7, SHAPE),
    ("ldy", 7, SHAPE), ("xs_off", -1, ARG), ("ws_off", 1 << 62, SHAPE), ("activation", 11, ARG),
    ("has_bias", 2, ARG), ("has_residual", 3, ARG), ("reserved", 1, ARG)])
def test_linear_int8_refusals(field, value, status):
    p = cf.make_linear_int8_problem(4, 8, 40, bias=True)
    setattr(p, field, value)
    assert int8(p) == status
    n = ctypes.c_uint64()
    assert cf.lib().linear_int8_scratch_size(ctypes.byref(p), 1, ctypes.byref(n)) == status
    with pytest.raises(cf.ConvError):
        cf.linear_int8_describe_variant(p, "f16")


def test_null_pointers_and_types():
    p = NORM()
    for dt in (3, -1):
        assert norm(p, dt) == norm_back(p, dt) == ARG
        assert drop(cf.make_dropout_problem(4, 8, 0.5), dt) == ARG
        assert quant(cf.make_quantize_problem(4, 8), dt) == ARG
        assert int8(cf.make_linear_int8_problem(4, 8, 8), dt) == ARG
    for name in ("x", "r", "w", "b", "y", "mean", "rstd"):  # mean without rstd, and the reverse
        assert norm(p, **{name: None}) == ARG, name
    for name in ("s", "w", "mean", "rstd", "dy"):
        assert norm_back(p, **{name: None}) == ARG, name
    assert norm_back(p, dx=None, dr=None, dw=None, db=None) == ARG  # nothing asked for
    q = cf.make_layer_norm_problem(4, 40, weight=False, bias=False)
    assert norm_back(q, dr=None, db=None) == ARG  # dw of no weight
    assert norm_back(q, dr=None, dw=None) == ARG  # db of no bias
    assert norm_back(q, dw=None, db=None) == ARG  # dr of no residual
    for name in ("x", "r", "y"):
        assert drop(cf.make_dropout_problem(4, 8, 0.5, residual=True), **{name: None}) == ARG
    for name in ("x", "q", "scale"):
        assert quant(cf.make_quantize_problem(4, 8), **{name: None}) == ARG
    p = cf.make_linear_int8_problem(4, 8, 40, bias=True, residual="after")
    for name in ("x", "xs", "w", "ws", "b", "r", "y"):
        assert int8(p, **{name: None}) == ARG, name


def test_no_rows():
    """m = 0: operands of m rows may be null."""
    p = cf.make_layer_norm_problem(0, 40, residual=True)
    none = dict(x=None, r=None, y=None, s=None, mean=None, rstd=None)
    assert norm(p, **none) == cf.CONV_OK
    assert norm_back(p, s=None, mean=None, rstd=None, dy=None, ds=None, dx=None, dr=None) == cf.CONV_OK
    assert norm(p, w=None, **none) == ARG
    assert drop(cf.make_dropout_problem(0, 8, 0.5), x=None, y=None) == cf.CONV_OK
    assert quant(cf.make_quantize_problem(0, 8), x=None, q=None, scale=None) == cf.CONV_OK
    assert int8(cf.make_linear_int8_problem(0, 8, 40), x=None, xs=None, y=None) == cf.CONV_OK


def test_misaligned_operands():
    for name in ("x", "r", "w", "b", "y", "s", "mean", "rstd", "step"):
        assert norm(NORM(), "f32", **{name: at(12) + 2}) == ARG, name
    for name in ("s", "w", "mean", "rstd", "dy", "ds", "dx", "dr", "dw", "db", "step"):
        assert norm_back(NORM(), "f32", **{name: at(12) + 2}) == ARG, name
    p = cf.make_dropout_problem(4, 40, 0.5, residual=True)
    for name in ("x", "r", "y"):
        assert drop(p, **{name: at(12) + 1}) == ARG, name
    assert drop(p, step=at(12) + 4) == ARG
    assert quant(cf.make_quantize_problem(4, 40), scale=at(12) + 2) == ARG
    assert quant(cf.make_quantize_problem(4, 40), q=at(12) + 1) == cf.CONV_OK  # bytes
    p = cf.make_linear_int8_problem(4, 8, 40, bias=True, residual="before")
    for name in ("xs", "ws", "b", "r", "y"):
        assert int8(p, **{name: at(12) + 1}) == ARG, name
    assert int8(p, x=at(12) + 1, w=at(13) + 3) == cf.CONV_OK


def test_overlaps():
    p = NORM()
    assert norm(p, y=at(0)) == norm(p, y=at(1)) == norm(p, s=at(1)) == cf.CONV_OK  # in place
    assert norm(p, y=at(0) + 2) == OVERLAP and norm(p, s=at(1) + 160) == OVERLAP
    assert norm(p, y=at(0), s=at(0)) == OVERLAP  # both outputs in one place
    for name in ("w", "b"):
        assert norm(p, y=at({"w": 2, "b": 3}[name])) == OVERLAP
    assert norm(p, mean=at(0)) == norm(p, rstd=at(6)) == norm(p, y=at(8)) == OVERLAP
    assert norm(NORM(ldx=48), y=at(0)) == OVERLAP  # another stride
    assert norm(NORM(ldx=80, ldy=80), y=at(0) + 80) == cf.CONV_OK  # two halves of wide rows
    assert norm(NORM(ldx=80, ldy=80), y=at(0) + 78) == OVERLAP
    assert norm_back(p, dx=at(4)) == norm_back(p, dx=at(5)) == norm_back(p, dr=at(5)) == cf.CONV_OK
    assert norm_back(p, dx=at(4), dr=at(4)) == norm_back(p, dx=at(0)) == OVERLAP
    assert norm_back(p, dw=at(1)) == norm_back(p, dw=at(10)) == norm_back(p, db=at(2)) == OVERLAP
    assert cf.layer_norm_backward_scratch_size(p, "f16") == 0
    assert norm_back(p, scratch=None, scratch_bytes=0) == cf.CONV_OK
    p = cf.make_layer_norm_problem(2000, 40, residual=True, drop=0.1)
    n = cf.layer_norm_backward_scratch_size(p, "f16")
    assert norm_back(p, scratch=at(4) - 256, scratch_bytes=n) == OVERLAP
    assert norm_back(p, scratch_bytes=n - 1) == SCRATCH
    assert norm_back(p, scratch=None) == norm_back(p, scratch=at(9) + 16) == ARG
    p = cf.make_dropout_problem(4, 40, 0.5, residual=True)
    assert drop(p, y=at(0)) == drop(p, y=at(1)) == cf.CONV_OK
    assert drop(p, y=at(0) + 2) == drop(p, y=at(3)) == OVERLAP
    assert cf.dropout_backward_check(p, "f16", at(0), at(0)) == cf.CONV_OK
    assert cf.dropout_backward_check(p, "f16", at(0), at(0) + 80) == OVERLAP
    p = cf.make_quantize_problem(4, 40)
    assert quant(p, q=at(0)) == quant(p, scale=at(1)) == quant(p, scale=at(0)) == OVERLAP
    p = cf.make_linear_int8_problem(4, 8, 40, bias=True, residual="before")
    assert int8(p, y=at(5)) == cf.CONV_OK
    for i in (0, 1, 2, 3, 4):
        assert int8(p, y=at(i)) == OVERLAP, i
    assert int8(p, y=at(5) + 2) == OVERLAP


def test_scratch_is_shape_only():
    """The same figures for every type and every mask; int8 products need none unless they
    are split or their rows are packed."""
    for m, n in ((1, 8), (100, 4096), (3, 100_000), (0, 7)):
        got = {cf.layer_norm_backward_scratch_size(cf.make_layer_norm_problem(m, n, drop=d), t)
               for d in (0.0, 0.5) for t in ("f32", "f16", "bf16")}
        assert len(got) == 1
    assert cf.linear_int8_scratch_size(cf.make_linear_int8_problem(8192, 4096, 4096), "f32") == 0
    assert "split" in cf.linear_int8_describe_variant(cf.make_linear_int8_problem(64, 256, 4096), "f16")
    assert cf.linear_int8_scratch_size(cf.make_linear_int8_problem(64, 256, 4096), "f16") > 0


def test_seeds_are_64_bits():
    for bad in (-1, 1 << 64):
        with pytest.raises(ValueError):
            cf.make_dropout_problem(1, 1, 0.5, seed=bad)
        with pytest.raises(ValueError):
            cf.make_layer_norm_problem(1, 1, offset=bad)


def test_generator_against_its_published_answers():
    """Known answers of Philox4x32-10, as its authors publish them."""
    for counter, key, want in (
            ([0] * 4, [0] * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
            ([mask.M32] * 4, [mask.M32] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
             "d16cfe09 94fdcceb 5001e420 24126ea1")):
        assert " ".join("%08x" % int(w) for w in mask.philox(counter, key)) == want


def test_mask_reference():
    assert mask.threshold(0.0) == 0 and mask.threshold(1.0) == 65536
    assert mask.threshold(2.0 ** -18) == 0 and mask.threshold(0.5) == 32768
    keep = mask.keeps(200, 801, 0.3, seed=5, offset=9)
    # 160200 draws: the share kept is within 6 standard deviations of 0.7
    assert abs(keep.mean() - 0.7) < 6 * math.sqrt(0.21 / keep.size)
    assert np.array_equal(keep[:50, :100], mask.keeps(50, 100, 0.3, seed=5, offset=9))
    assert not np.array_equal(keep, mask.keeps(200, 801, 0.3, seed=5, offset=10))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_planners_under_sanitizers(tmp_path):
    exe = str(tmp_path / "driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "rows_sanitize_driver.cpp"),
           *(os.path.join(CSRC, f) for f in ("rows_plan.cpp", "linear_int8_plan.cpp",
                                             "linear_plan.cpp", "conv_plan.cpp")), "-o", exe]
    built = subprocess.run(cmd, capture_output=True, text=True)
    if built.returncode and "cannot find -l" in built.stderr:
        pytest.skip("no sanitizer runtime")
    assert built.returncode == 0, built.stderr[-2000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout[-500:] + run.stderr[-2000:]
