"""Host logic of the rotary positions and the key/value cache: argument checks before any CUDA call, the binding's
refusals, and the frequencies. No compute call is made."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import bit_diffusion_transformer_svdquant_b200 as svdq
from bit_diffusion_transformer_svdquant_b200 import _lib, build
from oracle import heads as oracle

BASE = 1 << 40


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def _heads(at, n=6, rows=5, D=40, out=None, **kw):
    """A contiguous [rows, n, D] tensor at a fake address."""
    h = _lib.SvdqHeads(x=BASE + (at << 24), st=n * D, sh=D, heads=n)
    if out is not None:
        h.out, h.ot, h.oh = BASE + (out << 24), n * D, D
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def _set(obj, changes):
    for k, v in changes.items():
        *path, last = k.split("__")
        o = obj
        for p in path:
            o = getattr(o, p)
        if last == "axis_pairs":
            v = (ctypes.c_int * 4)(*v)
        setattr(o, last, v)
    return obj


def _args(**changes):
    """A well-formed rotation of q and k, 5 rows of 6 and 2 heads of 40."""
    a = _lib.SvdqHeadsArgs(samples=1, rows_per_sample=5, D=40, q=_heads(0, out=1), k=_heads(2, 2, out=3))
    a.rope = _lib.SvdqRope(dim=16, axes=2, axis_pairs=(ctypes.c_int * 4)(5, 3, 0, 0), amplitude=1.0, turns=BASE + (20 << 24),
                           positions=BASE + (21 << 24), pt=2)
    return _set(a, changes)


BAD = [
    (dict(D=39), 2), (dict(D=0), 2), (dict(D=258), 2), (dict(samples=-1), 1), (dict(x_f32=2), 1), (dict(out_f32=-1), 1),
    (dict(rope__dim=0), 1), (dict(rope__dim=15), 1), (dict(rope__dim=42), 1), (dict(rope__axes=0), 1), (dict(rope__axes=5), 1),
    (dict(rope__axis_pairs=(5, 4, 0, 0)), 1), (dict(rope__axis_pairs=(8, 0, 0, 0)), 1), (dict(rope__half=2), 1),
    (dict(rope__inverse=2), 1), (dict(rope__positions_i64=3), 1), (dict(rope__turns=None), 1), (dict(rope__positions=None), 1),
    (dict(rope__positions=BASE + 2), 2), (dict(rope__positions=BASE + 4, rope__positions_i64=1), 2), (dict(rope__pt=-1), 1),
    (dict(q__heads=0), 1), (dict(q__heads=5000), 1), (dict(k__heads=-1), 1), (dict(q__x=None), 1), (dict(q__out=None), 1),
    (dict(q__x=BASE + 1), 2), (dict(x_f32=1, q__x=BASE + 2), 2), (dict(q__st=-1), 1), (dict(k__sh=1 << 38), 1),
    (dict(q__norm__kind=3), 1), (dict(q__norm__kind=1, q__norm__eps=-1.0), 1),
    (dict(k__norm__kind=2, k__norm__eps=float("nan")), 1), (dict(q__norm__kind=1, q__norm__weight=BASE + 1), 2),
    (dict(v__heads=2), 1),                                            # v belongs to the cache
    (dict(q__ot=39), 1), (dict(q__oh=39), 1),                         # an output that overlaps itself
    (dict(q__out=BASE + 80), 1), (dict(q__out=BASE, q__ot=241), 1),   # over its input, but not its input
    (dict(q__out=BASE + (2 << 24)), 1), (dict(k__out=BASE + (1 << 24) + 64), 1), (dict(k__out=BASE), 1),
    (dict(q__out=BASE, out_f32=1), 1),                                # in place in another type
]


@pytest.mark.parametrize("changes,status", BAD)
def test_rotary_refusals(L, changes, status):
    assert L.svdq_rotary(ctypes.byref(_args(**changes)), None) == status, L.svdq_last_error()


QKV = dict(q__st=400, k__st=400, q__x=BASE, k__x=BASE + 480)
WELL = [{}, dict(k__heads=0), dict(q__out=BASE), dict(rope__dim=40, rope__axes=1, rope__axis_pairs=(20, 0, 0, 0)),
        QKV, dict(QKV, q__out=BASE, q__ot=400, k__out=BASE + 480, k__ot=400),       # slices of one buffer, in place
        dict(QKV, q__out=BASE, q__ot=400, k__out=BASE + 640, k__ot=400),            # beside the inputs' columns
        dict(q__oh=200, q__ot=40), dict(D=38, q__st=300, k__st=300), dict(q__sh=0)]


@pytest.mark.parametrize("changes", WELL)
def test_rotary_well_formed(L, changes):
    if torch.cuda.is_available():
        pytest.skip("fake addresses: CPU only")
    assert L.svdq_rotary(ctypes.byref(_args(**changes)), None) == 3, L.svdq_last_error()


def test_no_rows_is_no_work(L):
    for empty in (dict(samples=0), dict(rows_per_sample=0)):
        assert L.svdq_rotary(ctypes.byref(_args(**empty, q__x=None, q__out=None)), None) == 0
    assert L.svdq_rotary(None, None) == 1


def _cache(**changes):
    c = _lib.SvdqKvCache(pages=7, page_size=16, heads=2, D=40, format=0)
    for i in range(2):
        c.codes[i], c.scales[i] = BASE + ((30 + i) << 24), BASE + ((32 + i) << 24) + 1
    return _set(c, changes)


def _write_args(**changes):
    a = _args(k__out=None, k__ot=0, k__oh=0, v=_heads(5, 2))
    return _set(a, changes)


SLOTS = ctypes.c_void_p(BASE + (40 << 24))


def _write(L, cache=None, slots=SLOTS, i64=0, **changes):
    return L.svdq_kv_write(ctypes.byref(cache or _cache()), ctypes.byref(_write_args(**changes)), slots, i64, None)


@pytest.mark.parametrize("changes,status", [
    (dict(pages=0), 1), (dict(page_size=0), 1), (dict(heads=0), 1), (dict(heads=5000), 1), (dict(D=4), 2), (dict(D=44), 2),
    (dict(D=264), 2), (dict(format=2), 1), (dict(pages=(1 << 31) - 1, page_size=1 << 20), 1)])
def test_caches_refused(L, changes, status):
    c = _cache(**changes)
    assert _write(L, c) == status
    assert L.svdq_kv_read(ctypes.byref(c), SLOTS, 4, 4, SLOTS, 1, 4, SLOTS, 80, 40, SLOTS, 80, 40, 0, None) == status


def test_cache_buffers_refused(L):
    for field, i, value, status in (("codes", 0, None, 1), ("scales", 1, None, 1), ("codes", 1, BASE + 8, 2)):
        c = _cache()
        getattr(c, field)[i] = value
        assert _write(L, c) == status


@pytest.mark.parametrize("changes,status", [
    (dict(k__heads=3), 1), (dict(v__heads=1), 1), (dict(D=32, rope__dim=16), 1), (dict(v__norm__kind=1), 1),
    (dict(k__x=None), 1), (dict(v__x=None), 1), (dict(q__out=None), 1), (dict(rope__dim=17), 1),
    (dict(q__out=BASE + (5 << 24)), 1), (dict(q__out=BASE + (2 << 24) + 80), 1)])
def test_write_refusals(L, changes, status):
    assert _write(L, **changes) == status, L.svdq_last_error()


def test_write_slots_and_rows(L):
    assert _write(L, slots=None) == 1
    assert _write(L, i64=2) == 1
    assert _write(L, slots=ctypes.c_void_p(BASE + 2)) == 2
    assert _write(L, slots=ctypes.c_void_p(BASE + 4), i64=1) == 2
    assert _write(L, samples=0, slots=None) == 0
    if not torch.cuda.is_available():
        assert _write(L) == 3 and _write(L, q__heads=0) == 3 and _write(L, rope__dim=0) == 3 and _write(L, i64=1) == 3


def _read(L, c=None, table=SLOTS, ld=4, width=4, offsets=SLOTS, samples=3, rows=9, k=50, kr=80, kh=40, v=51, vr=80, vh=40, dt=0):
    at = lambda i: None if i is None else ctypes.c_void_p(BASE + int(i * (1 << 24)))
    return L.svdq_kv_read(ctypes.byref(c or _cache()), table, ld, width, offsets, samples, rows, at(k), kr, kh, at(v), vr, vh, dt,
                          None)


@pytest.mark.parametrize("changes,status", [
    (dict(offsets=None), 1), (dict(table=None), 1), (dict(samples=0), 1), (dict(rows=-1), 1), (dict(width=-1), 1),
    (dict(ld=3), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(dt=2), 1), (dict(kr=79), 1), (dict(vh=39), 1), (dict(kr=-80), 1),
    (dict(v=50), 1), (dict(k=50 + 2 ** -24), 2), (dict(table=ctypes.c_void_p(BASE + 2)), 2)])
def test_read_refusals(L, changes, status):
    assert _read(L, **changes) == status, L.svdq_last_error()


def test_read_well_formed(L):
    assert _read(L, rows=0, k=None, v=None) == 0
    if not torch.cuda.is_available():
        assert _read(L) == 3 and _read(L, dt=1) == 3 and _read(L, width=0, ld=0, table=None) == 3
        assert _read(L, kr=160, vr=160, v=50 + 160 / 2 ** 24) == 3      # keys and values in alternate columns
        assert _read(L, kr=40, kh=400, vr=40, vh=400) == 3              # heads outside


def test_structures_match_the_header(L, tmp_path):
    fields = {"svdq_rope": _lib.SvdqRope, "svdq_heads": _lib.SvdqHeads, "svdq_heads_args": _lib.SvdqHeadsArgs,
              "svdq_kv_cache": _lib.SvdqKvCache, "svdq_fp8b_weight": _lib.SvdqFp8bWeight, "svdq_fp8b_act": _lib.SvdqFp8bAct}
    lines = ['#include <stdio.h>', '#include "svdq.h"', "int main(void) {"]
    want = []
    for name, cls in fields.items():
        lines.append(f'  printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, *_ in cls._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Werror", "-I", os.path.dirname(_lib.HEADER), str(src), "-o",
                    str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == want


def test_packed_arguments_are_the_structure():
    """struct.pack of the fields in order gives the structure's bytes."""
    heads = tuple(range(1, 9)) + (3, 0, 1, 0.5, 1, 0, 11, 12)
    rope = (16, 1, 0, 2, 5, 3, 0, 0, 1.25, 1, 13, 14, 15, 16)
    raw = _lib._PACK_HEADS_ARGS(1, 2, 3, 0, 1, 0, *heads, *heads, *heads, *rope)
    a = _lib.SvdqHeadsArgs.from_buffer_copy(raw)
    assert (a.samples, a.rows_per_sample, a.D, a.x_f32, a.out_f32) == (1, 2, 3, 0, 1)
    for h in (a.q, a.k, a.v):
        assert (h.x, h.sb, h.st, h.sh, h.out, h.ob, h.ot, h.oh, h.heads) == (1, 2, 3, 4, 5, 6, 7, 8, 3)
        assert (h.norm.kind, h.norm.eps, h.norm.f32, h.norm.weight, h.norm.bias) == (1, 0.5, 1, 11, 12)
    r = a.rope
    assert (r.dim, r.half, r.inverse, r.axes, list(r.axis_pairs), r.amplitude, r.positions_i64, r.turns, r.positions, r.pb,
            r.pt) == (16, 1, 0, 2, [5, 3, 0, 0], 1.25, 1, 13, 14, 15, 16)


# ---------------------------------------------------------------- frequencies

def _rotary(**kw):
    """A Rotary whose table stays on the CPU."""
    r = svdq.Rotary.__new__(svdq.Rotary)
    r.dim, r.axes, r.layout, r.theta = sum(kw["axes"]), kw["axes"], "half", kw.get("theta", 10000.0)
    r.scaling = kw.get("scaling")
    return r


@pytest.mark.parametrize("axes,theta,scaling", [
    ([128], 10000.0, None), ([32, 32, 32, 32], 2000.0, None), ([40], 10000.0, {"kind": "linear", "factor": 8.0}),
    ([64, 32], 500000.0, {"kind": "ntk", "factor": 4.0}),
    ([80], 10000.0, {"kind": "yarn", "factor": 8.0, "length": 4096}),
    ([80], 10000.0, {"kind": "yarn", "factor": 8.0, "length": 4096, "beta_fast": 16.0, "beta_slow": 2.0, "amplitude": 1.0})])
def test_frequencies(axes, theta, scaling):
    got, amp = _rotary(axes=axes, theta=theta, scaling=scaling)._scaled()
    want, want_amp = oracle.frequencies(axes, theta, scaling)
    assert np.allclose(got, want, rtol=1e-14) and math.isclose(amp, want_amp)


@pytest.mark.parametrize("kw", [
    dict(dim=15), dict(dim=16, axes=[8, 6]), dict(dim=10, axes=[5, 5]), dict(dim=10, axes=[2] * 5), dict(dim=0),
    dict(dim=16, layout="split"), dict(dim=16, theta=0.0), dict(dim=16, theta=float("inf")), dict(dim=16, device="cpu"),
    dict(dim=16, scaling={"kind": "cubic", "factor": 2.0}), dict(dim=16, scaling={"kind": "linear"}),
    dict(dim=16, scaling={"kind": "linear", "factor": -1.0}), dict(dim=16, scaling={"kind": "linear", "factor": 2.0, "length": 9}),
    dict(dim=16, scaling={"kind": "yarn", "factor": 2.0}), dict(dim=2, scaling={"kind": "ntk", "factor": 2.0}),
    dict(dim=16, scaling={"kind": "yarn", "factor": 2.0, "length": 4096, "beta_fast": 1.0, "beta_slow": 1.0})])
def test_rotary_arguments_refused(kw):
    with pytest.raises(ValueError):
        svdq.Rotary(**kw)


def test_cpu_tensors_are_refused(L):
    x = torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        svdq.rotary(x, None, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        svdq.KvCache(4, 16, 2, 64, format="int8")
    with pytest.raises(svdq.SvdqError):
        svdq.KvCache(4, 16, 2, 60)
    with pytest.raises(ValueError, match="CUDA"):
        svdq.KvCache(4, 16, 2, 64, device="cpu")


# ---------------------------------------------------------------- which outputs share memory

def _bytes(at, dims, width):
    """The bytes of runs of `width` at `at` plus every sum of index x stride."""
    starts = np.array([at], dtype=np.int64)
    for stride, n in dims:
        starts = (starts[:, None] + stride * np.arange(n)).ravel()
    return starts, np.sort((starts[:, None] + np.arange(width)).ravel())


def test_slices_in_attention_layout_share_nothing(L):
    """q and k as slices of one [samples, 2, heads, rows, D] buffer, from inputs elsewhere and from slices of another."""
    if torch.cuda.is_available():
        pytest.skip("fake addresses: CPU only")
    B, T, H, D = 2, 5, 6, 40
    view = dict(ob=2 * H * T * D, ot=D, oh=T * D)
    both = {f"q__{k}": v for k, v in view.items()} | {f"k__{k}": v for k, v in view.items()}
    apart = dict(samples=B, q__sb=T * H * D, k__sb=T * H * D, k__st=H * D, k__heads=H, k__out=BASE + (1 << 24) + H * T * D * 2)
    assert L.svdq_rotary(ctypes.byref(_args(**both, **apart)), None) == 3, L.svdq_last_error()
    apart["k__out"] -= 2                                    # the first value of k is the last of q
    assert L.svdq_rotary(ctypes.byref(_args(**both, **apart)), None) == 1
    # rotated where they lie: the same slices are the inputs
    inputs = {f"{t}__{i}": v for t in "qk" for i, v in (("sb", view["ob"]), ("st", D), ("sh", T * D))}
    apart |= inputs | dict(k__out=BASE + (1 << 24) + H * T * D * 2, q__x=BASE + (1 << 24),
                           k__x=BASE + (1 << 24) + H * T * D * 2)
    assert L.svdq_rotary(ctypes.byref(_args(**both, **apart)), None) == 3, L.svdq_last_error()


def test_overlaps_are_those_of_the_bytes(L):
    """Small tensors of any strides and distances: refused exactly where two places of an output, or an output and another
    tensor, share a byte (an output that is its own input apart)."""
    if torch.cuda.is_available():
        pytest.skip("fake addresses: CPU only")
    rng = np.random.default_rng(5)
    D, seen = 2, {1: 0, 3: 0}
    for trial in range(4000):
        B, T = int(rng.integers(1, 4)), int(rng.integers(1, 5))
        f32 = int(rng.integers(0, 2))
        a = _args(samples=B, rows_per_sample=T, D=D, x_f32=f32, out_f32=int(rng.integers(0, 2)), rope__dim=2, rope__axes=1,
                  rope__axis_pairs=(1, 0, 0, 0), rope__pt=1)
        nested = [int(i) for i in rng.permutation(3)]
        tensors = []
        for n, t in enumerate((a.q, a.k)):
            t.heads = int(rng.integers(1, 4))
            counts = [B, T, t.heads]
            for x, out in ((True, False), (False, True)):
                strides, unit = [0, 0, 0], D * int(rng.integers(1, 3))
                for i in nested:
                    strides[i] = unit
                    unit *= counts[i]
                if rng.random() < 0.5:
                    strides = [int(rng.integers(0, 3 * D * max(counts))) for _ in range(3)]
                size = 4 if (a.x_f32 if x else a.out_f32) else 2
                at = BASE + size * int(rng.integers(0, 60))
                if x:
                    t.x, (t.sb, t.st, t.sh) = at, strides
                else:
                    if rng.random() < 0.3:
                        at, strides = t.x, [t.sb, t.st, t.sh]
                    t.out, (t.ob, t.ot, t.oh) = at, strides
                tensors.append((n, out, at, strides, counts, size))
        places = [(n, out, *_bytes(at, [(s * size, c) for s, c in zip(st, counts)], D * size),
                   (at, size, tuple(s for s, c in zip(st, counts) if c > 1))) for n, out, at, st, counts, size in tensors]
        if any(p[2][0] % (4 if a.out_f32 else 2) for p in places if p[1]):
            continue
        refuse = any(out and len(np.unique(b)) != len(b) for _, out, _, b, _ in places)
        for i, (n, out, _, b, view) in enumerate(places):
            for j, (m, other_out, _, c, other) in enumerate(places):
                if out and i != j and not (n == m and not other_out and view == other):
                    refuse |= len(np.intersect1d(b, c)) > 0
        got = L.svdq_rotary(ctypes.byref(a), None)
        assert got == (1 if refuse else 3), (trial, L.svdq_last_error(), tensors)
        seen[got] += 1
    assert min(seen.values()) > 200, seen


NORMED = dict(q__norm__kind=2, q__norm__eps=1e-6, q__norm__f32=1, k__norm__kind=1, k__norm__eps=1e-6)
OUT = BASE + (1 << 24)  # q's output: 5 rows of 6 heads of 40 bf16 values, 2400 bytes


@pytest.mark.parametrize("changes", [
    dict(rope__positions=OUT), dict(rope__positions=OUT + 2396), dict(rope__positions=OUT - 36), dict(rope__turns=OUT - 56),
    dict(rope__turns=OUT + 2392), dict(NORMED, q__norm__weight=OUT + 2396), dict(NORMED, q__norm__bias=OUT - 156),
    dict(NORMED, k__norm__weight=OUT + 2398)])
def test_outputs_over_what_is_read_are_refused(L, changes):
    """Positions, frequencies and the norms' vectors whose first or last element lies in q's output."""
    assert L.svdq_rotary(ctypes.byref(_args(**changes)), None) == 1
    assert b"overlaps" in L.svdq_last_error()
    assert _write(L, **changes) == 1 and b"overlaps" in L.svdq_last_error()


@pytest.mark.parametrize("changes", [
    dict(rope__positions=OUT + 2400), dict(rope__positions=OUT - 40), dict(rope__turns=OUT - 64), dict(rope__turns=OUT + 2400),
    dict(NORMED, q__norm__weight=OUT + 2400), dict(NORMED, q__norm__bias=OUT - 160), dict(NORMED, k__norm__weight=OUT - 80),
    dict(q__norm__weight=OUT),                                        # no norm: its vectors are not read
    dict(q__ot=480, rope__positions=OUT + 480, rope__pt=240)])        # positions behind each row's heads
def test_outputs_beside_what_is_read_are_taken(L, changes):
    if torch.cuda.is_available():
        pytest.skip("fake addresses: CPU only")
    assert L.svdq_rotary(ctypes.byref(_args(**changes)), None) == 3, L.svdq_last_error()
    assert _write(L, **changes) == 3, L.svdq_last_error()


CODES, SCALES = 7 * 16 * 2 * 40, 7 * 16 * 2  # bytes of a plane


def test_a_cache_over_what_the_write_touches_is_refused(L):
    k0, s1 = BASE + (30 << 24), BASE + (33 << 24) + 1
    for changes in (dict(k__x=k0 + CODES - 2), dict(v__x=k0), dict(q__out=k0 + CODES - 2), dict(q__x=k0), dict(v__x=s1 + SCALES - 1),
                    dict(rope__positions=k0 + 4)):
        assert _write(L, **changes) == 1 and b"overlaps" in L.svdq_last_error(), changes
    assert _write(L, slots=ctypes.c_void_p(k0 + CODES - 4)) == 1 and b"the slots" in L.svdq_last_error()
    assert _write(L, slots=ctypes.c_void_p(k0 - 32), i64=1) == 1 and b"the slots" in L.svdq_last_error()
    for field, i, at in (("codes", 1, k0), ("codes", 1, k0 + CODES - 16), ("scales", 0, k0 + 5), ("scales", 1, BASE + (32 << 24) + SCALES)):
        c = _cache()
        getattr(c, field)[i] = at
        assert _write(L, c) == 1 and b"the cache's" in L.svdq_last_error(), (field, i)
    if not torch.cuda.is_available():
        c = _cache()
        c.codes[1], c.scales[0], c.scales[1] = k0 + CODES, k0 + 2 * CODES, k0 + 2 * CODES + SCALES   # one buffer, no gaps
        assert _write(L, c, v__x=k0 - 800, q__out=k0 + 2 * CODES + 2 * SCALES) == 3, L.svdq_last_error()


def test_values_over_what_the_read_touches_are_refused(L):
    """9 rows of 2 heads of 40 (1440 bytes) over the cache's planes, the table and the offsets."""
    at = lambda b: (b - BASE) / 2 ** 24
    k0, s1 = BASE + (30 << 24), BASE + (33 << 24) + 1
    for changes in (dict(k=at(k0 - 1438)), dict(v=at(k0 + CODES - 2)), dict(k=at(s1 + SCALES - 1)), dict(v=at(SLOTS.value + 44)),
                    dict(k=at(SLOTS.value - 1438))):
        assert _read(L, **changes) == 1 and b"overlaps" in L.svdq_last_error(), changes
    far = ctypes.c_void_p(BASE + (60 << 24))
    assert _read(L, offsets=far, k=60 + 12 / 2 ** 24) == 1 and b"the offsets" in L.svdq_last_error()
    if not torch.cuda.is_available():
        assert _read(L, k=at(k0 - 1440), v=at(k0 + CODES), offsets=far) == 3, L.svdq_last_error()
        assert _read(L, offsets=far, k=60 + 16 / 2 ** 24) == 3, L.svdq_last_error()
        assert _read(L, table=SLOTS, offsets=far, width=0, ld=0, k=40) == 3, L.svdq_last_error()
