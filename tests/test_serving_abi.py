"""Refusals of the serving entry points, on the host before anything is
launched (the pointers are fakes that are never touched), and the binding's own
checks."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from exact_attention_28_gb300 import build, ops  # noqa: E402

INV, UNS, MIS = ops.FA_ERR_INVALID_ARG, ops.FA_ERR_UNSUPPORTED, ops.FA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.load_library()


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def doubles(n, value=0.5, at=None):
    a = (ctypes.c_double * n)(*([value] * n))
    if at is not None:
        a[at] = math.nan
    return a


def ints(n, value=0):
    return (ctypes.c_int * n)(*([value] * n))


TABLES = dict(table=0x10000, ctx=0x20000, new=0x30000, free=0x40000, seq=0x50000, start=0x60000, slots=0x70000,
              pos=0x80000, counts=0x90000, B=2, max_blocks=4, bs=16, num_free=3, tokens=5)


@pytest.mark.parametrize("kw,expected", [
    *[({k: 0}, INV) for k in ("table", "ctx", "new", "free", "seq", "start", "slots", "pos", "counts")],
    *[({k: 0x10002}, MIS) for k in ("table", "ctx", "new", "free", "seq", "start", "slots", "pos", "counts")],
    (dict(B=0), INV), (dict(B=16385), INV), (dict(max_blocks=0), INV), (dict(num_free=-1), INV),
    (dict(seq=0x20000), INV), (dict(start=0x30004), INV), (dict(table=0x40000), INV), (dict(slots=0x80004), INV),  # overlaps
    (dict(counts=0x5fffc), INV),
    (dict(tokens=-1), INV), (dict(tokens=(1 << 30) + 1), INV), (dict(bs=48), UNS), (dict(bs=8), UNS), (dict(max_blocks=1 << 28, bs=16), INV),
])
def test_block_tables_refusals(lib, kw, expected):
    a = dict(TABLES, **kw)
    assert lib.fa_block_tables(*[a[k] or None for k in ("table", "ctx", "new", "free", "seq", "start", "slots", "pos",
                                                         "counts")],
                               a["B"], a["max_blocks"], a["bs"], a["num_free"], a["tokens"], None) == expected


ROPE = dict(q=0x10000, qs=None, qo=0x20000, qos=None, Hq=4, k=0x30000, ks=None, ko=0x40000, kos=None, Hk=2,
            pos=0x50000, pa=8, pb=0, B=1, N=8, d=64, rot=64, axes=1, freq=doubles(32), axis=ints(32), inter=0, inv=0)


@pytest.mark.parametrize("kw,expected", [
    (dict(q=0), INV), (dict(qo=0), INV), (dict(k=0), INV), (dict(ko=0), INV), (dict(pos=0), INV),
    (dict(Hk=0), INV),                                    # K given, but no heads
    (dict(Hq=0), INV), (dict(Hk=-1), INV), (dict(B=0), INV), (dict(N=0), INV), (dict(B=1 << 16, N=1 << 16), INV),
    (dict(d=96), UNS), (dict(rot=0), UNS), (dict(rot=24), UNS), (dict(rot=80), UNS), (dict(rot=128), UNS),
    (dict(axes=0), INV), (dict(axes=5), INV), (dict(freq=None), INV), (dict(freq=doubles(32, math.inf)), INV),
    (dict(freq=doubles(32, at=31)), INV), (dict(axis=ints(32, 1)), INV), (dict(axis=ints(32, -1)), INV),
    (dict(q=0x10008), MIS), (dict(qo=0x20002), MIS), (dict(ko=0x40004), MIS), (dict(pos=0x50002), MIS),
    (dict(qs=strides(0, 64, 260)), MIS), (dict(kos=strides(1024, 512, 68)), MIS),
    (dict(qs=strides(0, -64, 64)), INV), (dict(qos=strides(2048, 0, 64)), INV),   # heads written on one another
    (dict(qos=strides(2048, 512, 32)), INV), (dict(pa=-1), INV), (dict(pb=-8), INV),
])
def test_rope_refusals(lib, kw, expected):
    a = dict(ROPE, **kw)
    assert lib.fa_rope(a["q"] or None, a["qs"], a["qo"] or None, a["qos"], a["Hq"], a["k"] or None, a["ks"],
                       a["ko"] or None, a["kos"], a["Hk"], a["pos"] or None, a["pa"], a["pb"], a["B"], a["N"], a["d"],
                       a["rot"], a["axes"], a["freq"], a["axis"], a["inter"], a["inv"], None) == expected


APPEND = dict(q=0x10000, qs=None, qo=0x20000, qos=None, Hq=4, k=0x30000, ks=None, v=0x40000, vs=None, Hkv=2,
              kc=0x50000, vc=0x60000, kind=1, kd=0x70000, vd=0x80000, slots=0x90000, pos=0xa0000, pa=8, T=8, blocks=4,
              bs=16, d=64, rot=64, axes=1, freq=doubles(32), axis=None, inter=0)


@pytest.mark.parametrize("kw,expected", [
    *[({k: 0}, INV) for k in ("q", "qo", "k", "v", "kc", "vc", "kd", "vd", "slots", "pos")],
    *[({k: 0x10008}, MIS) for k in ("q", "qo", "k", "v", "kc", "vc")],
    *[({k: 0x10002}, MIS) for k in ("kd", "vd", "slots", "pos")],
    (dict(Hq=0), INV), (dict(Hkv=0), INV), (dict(T=0), INV), (dict(blocks=0), INV), (dict(kind=2), INV),
    (dict(blocks=1 << 28), INV), (dict(bs=24), UNS), (dict(d=32), UNS), (dict(rot=8), UNS), (dict(axes=9), INV),
    (dict(freq=None), INV), (dict(ks=strides(130, 64)), MIS), (dict(qos=strides(0, 64)), INV), (dict(pa=-1), INV),
])
def test_append_refusals(lib, kw, expected):
    a = dict(APPEND, **kw)
    assert lib.fa_paged_append(a["q"] or None, a["qs"], a["qo"] or None, a["qos"], a["Hq"], a["k"] or None, a["ks"],
                               a["v"] or None, a["vs"], a["Hkv"], a["kc"] or None, a["vc"] or None, a["kind"],
                               a["kd"] or None, a["vd"] or None, a["slots"] or None, a["pos"] or None, a["pa"],
                               a["T"], a["blocks"], a["bs"], a["d"], a["rot"], a["axes"], a["freq"], a["axis"],
                               a["inter"], None) == expected


DECODE = dict(q=0x10000, qs=None, kc=0x20000, vc=0x30000, kind=1, kd=0x40000, vd=0x50000, table=0x60000, seq=0x70000,
              o=0x80000, os=None, lse=0x90000, B=2, Hq=4, Hkv=2, Nq=1, max_blocks=4, blocks=8, bs=16, d=64,
              scale=0.125, causal=0, ws=0x100000, nbytes=1 << 30)


@pytest.mark.parametrize("kw,expected", [
    *[({k: 0}, INV) for k in ("q", "kc", "vc", "kd", "vd", "table", "seq", "o", "lse", "ws")],
    *[({k: 0x10008}, MIS) for k in ("q", "kc", "vc", "o")],
    *[({k: 0x10002}, MIS) for k in ("kd", "vd", "table", "seq", "lse")],
    (dict(ws=0x100010), MIS), (dict(nbytes=0), INV), (dict(B=0), INV), (dict(Hq=0), INV), (dict(Hkv=0), INV),
    (dict(Hq=5), INV), (dict(Nq=0), INV), (dict(Nq=17), UNS), (dict(d=96), UNS), (dict(bs=8), UNS),
    (dict(max_blocks=0), INV), (dict(blocks=0), INV), (dict(scale=math.nan), INV), (dict(kind=-1), INV),
    (dict(qs=strides(4, 64, 64)), MIS), (dict(os=strides(256, 0, 64)), INV), (dict(max_blocks=1 << 27), INV),
    (dict(B=1 << 20, Hq=1 << 12), INV), (dict(B=1 << 19, Hkv=4, max_blocks=1 << 26), INV),
    (dict(B=1, Hq=1 << 16), INV), (dict(scale=3e38), INV), (dict(scale=-3e38), INV),
])
def test_decode_refusals(lib, kw, expected):
    a = dict(DECODE, **kw)
    assert lib.fa_decode_paged(a["q"] or None, a["qs"], a["kc"] or None, a["vc"] or None, a["kind"], a["kd"] or None,
                               a["vd"] or None, a["table"] or None, a["seq"] or None, a["o"] or None, a["os"],
                               a["lse"] or None, a["B"], a["Hq"], a["Hkv"], a["Nq"], a["max_blocks"], a["blocks"],
                               a["bs"], a["d"], a["scale"], a["causal"], a["ws"] or None, a["nbytes"], None) == expected


ROPE_ARGS = ("q", "qs", "qo", "qos", "Hq", "k", "ks", "ko", "kos", "Hk", "pos", "pa", "pb", "B", "N", "d", "rot", "axes",
             "freq", "axis", "inter", "inv")
APPEND_ARGS = ("q", "qs", "qo", "qos", "Hq", "k", "ks", "v", "vs", "Hkv", "kc", "vc", "kind", "kd", "vd", "slots", "pos",
               "pa", "T", "blocks", "bs", "d", "rot", "axes", "freq", "axis", "inter")
DECODE_ARGS = ("q", "qs", "kc", "vc", "kind", "kd", "vd", "table", "seq", "o", "os", "lse", "B", "Hq", "Hkv", "Nq",
               "max_blocks", "blocks", "bs", "d", "scale", "causal", "ws", "nbytes")


def no_gpu():
    return not torch.cuda.is_available()


# Outputs on other memory, and layouts beside them that are allowed: without a GPU those get as far as CUDA's error.
@pytest.mark.parametrize("fn,base,names,kw,refused", [
    ("fa_rope", ROPE, ROPE_ARGS, kw, refused) for kw, refused in [
        (dict(qos=strides(64, 64, 64)), True),                          # every head's rows on every other's
        (dict(qos=strides(2048, 64, 64)), True), (dict(qos=strides(2048, 448, 64)), True),
        (dict(qos=strides(0, 64, 192)), True),                          # 4 heads of 64 in rows of 192
        (dict(qos=strides(0, 64, 256)), False), (dict(qos=strides(64, 512, 64)), False),      # token-major; one batch
        (dict(B=2, qos=strides(1024, 512, 64)), True), (dict(B=2, qos=strides(64, 512, 128)), True),
        (dict(B=2, qos=strides(64, 1024, 128)), False),                 # batches side by side
        (dict(kos=strides(0, 64, 64)), True), (dict(Hk=1, kos=strides(0, 64, 64)), False),
        (dict(qo=0x40000), True),                                       # q's output is k's
        (dict(qo=0x10000), False), (dict(qo=0x10000, qos=strides(0, 64, 256)), True),         # in place, strides differ
        (dict(qo=0x10080), True), (dict(qo=0x30000), True), (dict(ko=0x10000), True), (dict(qo=0x3f800), True),
        (dict(ko=0x30000), False), (dict(qo=0x30000, qos=strides(0, 1024, 64)), True),
        (dict(ko=0x10000, qs=strides(0, 64, 256), kos=strides(0, 64, 512)), True),            # strided, first rows alike
        (dict(ko=0x10080, qs=strides(0, 1024, 128), kos=strides(0, 1024, 128)), False),       # rows between rows
    ]] + [("fa_paged_append", APPEND, APPEND_ARGS, kw, refused) for kw, refused in [
        (dict(qos=strides(64, 64)), True), (dict(qos=strides(256, 64)), False), (dict(qos=strides(64, 512)), False),
        (dict(qos=strides(64, 448)), True), (dict(vc=0x50000), True), (dict(vc=0x51000), True), (dict(vc=0x52000), False),
        (dict(vc=0x52000, kind=0), True), (dict(qo=0x10000), False), (dict(qo=0x10000, qos=strides(64, 512)), True),
        (dict(qo=0x30000), True), (dict(qo=0x50100), True), (dict(kc=0x8fff0), True), (dict(vc=0x40000), True),
    ]] + [("fa_decode_paged", DECODE, DECODE_ARGS, kw, refused) for kw, refused in [
        (dict(Nq=2, os=strides(512, 128, 64)), False), (dict(Nq=2, os=strides(512, 64, 64)), True),
        (dict(Nq=2, os=strides(64, 128, 512)), False), (dict(os=strides(64, 64, 64)), True),
        (dict(o=0x10000), False), (dict(o=0x10000, os=strides(256, 128, 64)), True),            # in place, strides differ
        (dict(o=0x10100), True), (dict(lse=0x80010), True), (dict(lse=0x70004), True), (dict(o=0x21000), True),
        (dict(ws=0x8ff00), True), (dict(lse=0x100100), True), (dict(vc=0x20000), False),      # one cache for both: read only
        (dict(o=0xfff00), True), (dict(seq=0x60000), False), (dict(ws=0x80200), True),
    ]])
def test_outputs_on_other_memory_are_refused(lib, fn, base, names, kw, refused):
    if not refused and not no_gpu():
        pytest.skip("the pointers are fakes")
    a = dict(base, **kw)
    pointers = {"q", "qo", "k", "ko", "v", "kc", "vc", "kd", "vd", "slots", "pos", "table", "seq", "o", "lse", "ws"}
    status = getattr(lib, fn)(*[(a[n] or None) if n in pointers else a[n] for n in names], None)
    assert status == (INV if refused else ops.FA_ERR_CUDA)


def test_decode_workspace_needs_no_gpu_and_checks_its_sizes(lib):
    assert ops.decode_paged_workspace(1, 32, 8, 1, 128) > 0
    for bad in ((0, 1, 1, 1, 64), (1, 3, 2, 1, 64), (1, 1, 1, 17, 64), (1, 1, 1, 1, 80)):
        with pytest.raises(ops.FAError):
            ops.decode_paged_workspace(*bad)


@pytest.mark.parametrize("kw", [
    dict(d=96), dict(d=64, rot=24), dict(d=64, rot=128), dict(d=64, sections=[16, 15]),
    dict(d=64, sections=[8, 8, 8, 4, 4]), dict(d=64, inv_freq=[1.0]), dict(d=64, inv_freq=[math.nan] * 32),
    dict(d=64, pair_axis=[4] * 32), dict(d=64, pair_axis=[-1] * 32), dict(d=64, sections=[32], pair_axis=[0] * 32),
])
def test_rotary_refusals(kw):
    with pytest.raises(ValueError):
        ops.Rotary(**kw)


def test_rotary_lays_out_axes_and_frequencies():
    r = ops.Rotary(64, base=100.0, rot=32, sections=[8, 4, 4])
    assert r.axes == 3 and r.pair_axis == (0,) * 8 + (1,) * 4 + (2,) * 4
    assert r.inv_freq[0] == 1.0 and abs(r.inv_freq[8] - 100.0 ** -0.5) < 1e-15


def test_binding_refuses_host_tensors_and_other_types():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        ops.fa_rope(q, None, pos, ops.Rotary(64))
    with pytest.raises(TypeError):
        ops.apply_rotary(q, q, pos, ops.Rotary(64))
    with pytest.raises(TypeError):
        ops.fa_paged_append(None, q[0], q[0], q, q, pos)
    with pytest.raises(TypeError):
        ops.fa_decode_paged(q, q, q, pos[None], pos[:1])
    with pytest.raises(TypeError):
        ops.fa_block_tables(pos[None], pos, pos, pos, 16, 1)


def test_a_call_makes_its_tensors_device_current(monkeypatch):
    """Two devices, of which the second one holds the tensors: the C call and its stream are that one's."""
    state = {"dev": 0}

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, state["dev"] = state["dev"], self.dev

        def __exit__(self, *exc):
            state["dev"] = self.before

    monkeypatch.setattr(ops, "_current_device", lambda: state["dev"])
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: 1000 + dev)
    monkeypatch.setattr(torch.cuda, "device", Device)
    calls = []

    def fn(*args):
        calls.append((state["dev"], args))
        return ops.FA_OK if args[0] != "bad" else INV

    ops._call(1, None, fn, "x", 2)
    ops._call(0, None, fn, "y")
    ops._call(1, 77, fn, "z")
    assert calls == [(1, ("x", 2, 1001)), (0, ("y", 1000)), (1, ("z", 77))] and state["dev"] == 0
    with pytest.raises(ops.FAError):
        ops._call(1, None, fn, "bad")
    assert state["dev"] == 0


def test_no_gpu_means_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    a = TABLES
    assert lib.fa_block_tables(*[a[k] for k in ("table", "ctx", "new", "free", "seq", "start", "slots", "pos", "counts")],
                               2, 4, 16, 3, 5, None) == ops.FA_ERR_CUDA
