"""What the library does when a CUDA launch is refused, on the CPU: its host code linked against a stand-in
for the CUDA runtime that records the launches and refuses the n-th."""
import concurrent.futures as futures
import ctypes
import os
import subprocess

import pytest

from block_sparse_attention_forecast_gb300 import build as _build

_build.build()

import block_sparse_attention_forecast_gb300.binding as sb  # noqa: E402

P = ctypes.c_void_p
TOO_LARGE = 720                                    # cudaErrorCooperativeLaunchTooLarge


def compiled(tmp, sources, fake="fake_cuda_runtime.cpp", extra=()):
    """A shared library of these files of csrc and the stand-in (fake=None: the CUDA runtime itself); calls
    into files left out are never made (their symbols are looked up when they are called)."""
    files = [os.path.join(_build.CSRC, s) for s in sources]
    if fake:
        files.append(os.path.join(os.path.dirname(os.path.abspath(__file__)), fake))
    objs = [os.path.join(tmp, os.path.basename(src) + ".o") for src in files]
    cmds = [[_build.nvcc()] + _build.ARCH + _build.FLAGS + list(extra) + ["-c", src, "-o", o] for src, o in zip(files, objs)]
    with futures.ThreadPoolExecutor() as ex:
        list(ex.map(lambda c: subprocess.run(c, check=True), cmds))
    lib = os.path.join(tmp, "host.so")
    subprocess.run([_build.nvcc()] + _build.ARCH + ["-shared", "-cudart", "none" if fake else "static", "-Xlinker", "-Bsymbolic",
                                                    "-Xlinker", "-z", "-Xlinker", "lazy", "-o", lib] + objs, check=True)
    dl = ctypes.CDLL(None)
    dl.dlopen.restype, dl.dlopen.argtypes = P, [ctypes.c_char_p, ctypes.c_int]
    handle = dl.dlopen(lib.encode(), os.RTLD_LAZY | os.RTLD_LOCAL)
    assert handle
    lib = ctypes.CDLL(lib, handle=handle)
    if fake:
        lib.fake_launch.restype = ctypes.c_char_p
    for name in ("sparda_evict_blocks", "sparda_kv4_evict_blocks", "sparda_kv4_decode_attn", "sparda_sparse_decode_attn_mass",
                 "sparda_device_error"):
        getattr(lib, name).argtypes = getattr(sb.lib, name).argtypes
    return lib


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return compiled(str(tmp_path_factory.mktemp("host")), ["api.cu", "evict.cu"])


def _names(lib):
    full = [lib.fake_launch(i).decode() for i in range(lib.fake_launches())]
    return [n[n.index("evict_"):n.index("_kernel")] for n in full]


def _evict(lib, kv4, in_place):
    s = sb.Shape(max_batch=2, max_ctx=4096)
    d = sb.Shape(max_batch=2, max_ctx=1024)
    mk = (lambda at: ctypes.byref(sb.c_layer_kv4(at, at << 1))) if kv4 else \
        (lambda at: ctypes.byref(sb.c_layer_kv(at, at << 1, at << 2, None, None, 0, 0)))
    fn = lib.sparda_kv4_evict_blocks if kv4 else lib.sparda_evict_blocks
    dst = (None,) * 4 if in_place else (ctypes.byref(d.c()), mk(1 << 40), P(1 << 21), P(1 << 23))
    return fn(ctypes.byref(s.c()), mk(1 << 32), P(1 << 20), P(1 << 22), *dst, 2, 8, 2, P(1 << 25), None)


ORDER = {True: ["evict_select", "evict_shift", "evict_join", "evict_length"], False: ["evict_select", "evict_move"]}


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kv4", [True, False])
def test_an_eviction_stops_at_a_refused_launch(lib, kv4, in_place):
    """Nothing is launched behind the refused one, the call reports it, and no error is left behind."""
    order = ORDER[in_place]
    for nth in range(len(order) + 1):
        lib.fake_reset(nth, TOO_LARGE)
        status = _evict(lib, kv4, in_place)
        assert status == (sb.ERR_CUDA if nth < len(order) else sb.OK), nth
        assert _names(lib) == order[:nth]
        assert lib.fake_last_error() == 0


def test_an_eviction_in_place_that_no_sm_can_hold_launches_nothing(tmp_path):
    lib = compiled(str(tmp_path), ["api.cu", "evict.cu"])
    lib.fake_reset(-1, 0)
    lib.fake_set_ctas_per_sm(0)
    for kv4 in (True, False):
        assert _evict(lib, kv4, True) == sb.ERR_CUDA and _names(lib) == [] and lib.fake_last_error() == 0
    lib.fake_set_ctas_per_sm(1)
    assert _evict(lib, True, True) == sb.OK and _names(lib) == ORDER[True]


@pytest.fixture(scope="module")
def attn(tmp_path_factory):
    return compiled(str(tmp_path_factory.mktemp("attn")), ["api.cu", "attn.cu", "kv4_attn.cu", "block_mass.cu"])


def _attend(lib, kv4, B, mass, H=16):
    s = sb.Shape(max_batch=B, max_ctx=4096, topk=62, heads_per_group=H)
    layer = ctypes.byref(sb.c_layer_kv4(1 << 32, 1 << 33) if kv4 else
                         sb.c_layer_kv(1 << 32, 1 << 33, 1 << 34, None, None, 0, 0))
    p = P(1 << 20)
    args = (ctypes.byref(s.c()), layer, p, p, p, p, B, p) + (P(1 << 22) if mass else None, p, 1 << 40, None)
    return (lib.sparda_kv4_decode_attn if kv4 else lib.sparda_sparse_decode_attn_mass)(*args)


@pytest.mark.parametrize("kv4", [True, False])
def test_no_block_mass_behind_a_refused_attention(attn, kv4):
    """The block mass is added from what the attention left: without the attention it must not be. 100
    sequences take the forms that leave it to a launch of its own."""
    kinds = lambda: ["mass" if b"block_mass" in attn.fake_launch(i) else "attention" for i in range(attn.fake_launches())]
    attn.fake_reset(-1, 0)
    assert _attend(attn, kv4, 100, True) == sb.OK and kinds() == ["attention", "mass"]
    for nth in (0, 1):
        attn.fake_reset(nth, 701)
        assert _attend(attn, kv4, 100, True) == sb.ERR_CUDA and kinds() == ["attention"] * nth
        assert attn.fake_last_error() == 0


def test_a_failed_question_to_the_runtime_is_not_kept(attn):
    """A call that cannot learn its kernel's registers fails and leaves no error behind; the next goes on."""
    attn.fake_reset(-1, 0)
    attn.fake_refuse_attributes(98)
    assert _attend(attn, True, 2, False, H=4) == sb.ERR_CUDA
    assert attn.fake_launches() == 0 and attn.fake_last_error() == 0
    assert _attend(attn, True, 2, False, H=4) == sb.OK and attn.fake_launches() == 1
