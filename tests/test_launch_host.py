"""The host code of the feature-row operators against a stand-in for the CUDA runtime: the library's own objects, linked
with tests/fake_cudart.c, so that launches can fail without a GPU and every call that was made can be looked at."""
import ctypes
import os
import subprocess

import pytest

LAUNCH, ATTRIBUTE, RECORD, WAIT = 1, 2, 3, 4
OK, CUDA = 0, 64
P = ctypes.c_void_p
HERE = os.path.dirname(os.path.abspath(__file__))


class Note(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("what", "a", "b", "c", "status")]


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from sparse_convolution_voxel_b200 import build
    build.build()
    at = tmp_path_factory.mktemp("fake")
    objs = [os.path.join(build.BUILD, f + ".cu.o") for f in ("embed", "norm")]
    subprocess.run(["gcc", "-O1", "-fPIC", "-c", os.path.join(HERE, "fake_cudart.c"), "-o", str(at / "fake.o")], check=True)
    # nothing but the entry points is exported: inline functions' variables (a thread's side stream, the device's
    # properties) would otherwise be one with those of the real library in this process
    (at / "exports").write_text("{ global: lat_*; fake_*; local: *; };")
    subprocess.run(["g++", "-shared", f"-Wl,--version-script={at / 'exports'}", "-Wl,--no-undefined", *objs,
                    str(at / "fake.o"), "-o", str(at / "libfake.so")], check=True)
    names = subprocess.run(["nm", "-D", "--defined-only", str(at / "libfake.so")], check=True, capture_output=True, text=True)
    assert all(line.split()[-1].startswith(("lat_", "fake_")) for line in names.stdout.splitlines())
    lib = ctypes.CDLL(str(at / "libfake.so"))
    I32, I64, SZ, F = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.lat_embed_wgrad_ws_bytes.restype, lib.lat_embed_wgrad_ws_bytes.argtypes = SZ, [I64, I64, I32]
    lib.lat_embed_wgrad.argtypes = [P, I32, I64, P, I64, I32, F, I64, P, I32, P, SZ, P, P]
    lib.lat_rms_norm_bwd.argtypes = [P, P, P, P, P, P, P, I64, I32, P, P, I32, P, SZ, P]
    return lib


def calls(lib, fail, f):
    """(status of f(), the calls that it made), call number `fail` failing."""
    lib.fake_reset(fail)
    status = f()
    out = ctypes.POINTER(Note)()
    n = lib.fake_notes(ctypes.byref(out))
    return status, [out[i] for i in range(n)]


@pytest.mark.parametrize("n,vocab,c", [(5000, 40000, 128), (300000, 50000, 128), (20000, 3000000, 8), (16383, 50257, 1024),
                                       (300, 40000, 128), (5000, 700, 128)])
def test_a_failed_call_leaves_no_work_behind_on_the_side_stream(fake, n, vocab, c):
    """Whichever call fails, a stream that was made to wait for the caller's is waited for before the entry point returns:
    else the zeros' kernel could still write a gradient that the caller frees, and a capture could not end."""
    stream = 0x77
    size = fake.lat_embed_wgrad_ws_bytes(n, vocab, c)

    def grad():
        return fake.lat_embed_wgrad(P(4096), 4, n, P(8192), vocab, c, 1.0, -1, P(1 << 30), 2, P(1 << 20), size, None,
                                    P(stream))

    status, made = calls(fake, -1, grad)
    assert status == OK
    large = n > 4096 and vocab * c * 4 >= 16 << 20
    assert any(m.what == LAUNCH and m.b != stream for m in made) == large, "the case takes the side stream"
    for fail in range(len(made)):
        status, got = calls(fake, fail, grad)
        assert status == CUDA, fail
        forks = [i for i, m in enumerate(got) if m.what == WAIT and m.a != stream and not m.status]
        if not forks:
            continue
        side = got[forks[0]].a
        joined = [i for i, m in enumerate(got) if m.what == WAIT and m.a == stream and not m.status]
        records = [i for i, m in enumerate(got) if m.what == RECORD and m.b == side and not m.status]
        if got[-1].status and got[-1].what in (RECORD, WAIT):
            continue  # the joining call itself is the one that failed
        assert len(joined) == 1 and len(records) == 1, f"call {fail} of {len(made)}"
        assert got[records[0]].a == got[joined[0]].b and records[0] < joined[0]
        assert all(m.b == stream for m in got[records[0]:] if m.what == LAUNCH)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_a_kernels_shared_memory_limit_does_not_change_between_calls(fake, dtype, q8):
    """Two host threads may call at once: a call that lowered the limit of a kernel that another one is about to launch
    with more would make that launch fail."""
    limits = {}
    h, h8 = (None, P(1 << 21)) if q8 else (P(1 << 21), None)
    for c in (8, 32, 40, 64, 72, 128, 256, 264, 512, 520, 1024, 1032, 2048, 4096, 5120, 8192, 8200, 12288, 16384):
        for dh in (None, P(1 << 22)):
            for dw in (None, P(1 << 23)):
                status, got = calls(fake, -1, lambda: fake.lat_rms_norm_bwd(
                    P(1 << 20), dh, h, h8, h8, P(4096), P(8192), 1000, c, P(1 << 24), dw, dtype, P(1 << 25), 1 << 30, None))
                assert status == OK
                for m in got:
                    if m.what == ATTRIBUTE:
                        limits.setdefault((m.a, m.b), set()).add(m.c)
                launched = [m for m in got if m.what == LAUNCH]
                assert len(launched) == (2 if dw else 1)
                most = max(v for (f, _), vs in limits.items() if f == launched[0].a for v in vs)
                assert launched[0].c <= most <= 232448 - 1024
    assert all(len(v) == 1 for v in limits.values()), sorted(map(sorted, limits.values()))
