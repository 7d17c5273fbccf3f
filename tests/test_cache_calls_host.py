"""Host paths of the paged-cache operators with a fake CUDA runtime (no GPU): which kernels a
call launches, and that a call that cannot launch them all is refused before it launches one.

The fake answers the runtime calls that libdan.so makes; it is loaded into a process of its own
ahead of the library, which finds the fake's functions in place of the runtime's.  It counts
the calls of each kind, fails the ones it is told to fail, and notes each launch's grid."""
import json
import os
import shutil
import subprocess
import sys

import pytest

from dit_adaln_norm_gb300 import build as dan_build
from dit_adaln_norm_gb300 import ops

OK, EINVAL, EUNSUP, EALIGN, EALIAS, ECUDA = range(6)

FAKE = r"""
#include <stddef.h>
#include <string.h>
enum { ENTRY, ENCODE, ATTRIBUTES, SET, LAUNCH, KINDS };
int count[KINDS], fail_at[KINDS], registers = 168, launches;
unsigned grids[64][4]; /* x, y, threads, bytes of shared memory */
static int failing(int kind) { return ++count[kind] == fail_at[kind]; }
static int encode(void) { return failing(ENCODE) ? 1 : 0; }
int cudaGetDevice(int *d) { return *d = 0; }
int cudaDeviceGetAttribute(int *v, int which, int d) { *v = which == 16 ? 152 : 232448; return 0; }
int cudaGetSymbolAddress(void **p, const void *s) { static unsigned word; *p = &word; return 0; }
int cudaGetDriverEntryPointByVersion(const char *n, void **p, unsigned v, unsigned long long fl, int *found)
{
    if (failing(ENTRY)) return 1;
    *p = (void *)encode;
    return *found = 0;
}
struct config { unsigned g[3], b[3]; size_t smem; };
int cudaLaunchKernelExC(const struct config *c, const void *f, void **args)
{
    if (failing(LAUNCH)) return 1;
    unsigned *at = grids[launches++];
    at[0] = c->g[0], at[1] = c->g[1], at[2] = c->b[0], at[3] = (unsigned)c->smem;
    return 0;
}
"""
# what needs a struct of the toolkit's header, or C++
ATTR = r"""
#include <cuda_runtime_api.h>
#include <new>
extern "C" int registers, count[], fail_at[];
extern "C" int throws = 0;
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int)
{
    if (++count[3] != fail_at[3]) return cudaSuccess;
    if (throws) throw std::bad_alloc();
    return cudaErrorUnknown;
}
extern "C" cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes *out, const void *)
{
    *out = cudaFuncAttributes();
    out->numRegs = registers;
    return ++count[2] == fail_at[2] ? cudaErrorUnknown : cudaSuccess;
}
"""
PRELUDE = r"""
import ctypes, json, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
I, P, F = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
lib.dan_window_attention.argtypes = [P, I, I, P, P, I, I, P, I, I, P, P] + [I] * 8 + [F, P, P, P, I, P]
lib.dan_window_attention_workspace.argtypes = [I] * 11
lib.dan_window_attention_workspace.restype = I
count, fail_at = ((ctypes.c_int * 5).in_dll(fake, n) for n in ("count", "fail_at"))
ENTRY, ENCODE, ATTRIBUTES, SET, LAUNCH = range(5)
def attention(N=500, S=4, H=32, Hkv=8, hd=128, M=64, page=64, window=1 << 20, sinks=0, chunk=1, max_q=None):
    max_q = N if max_q is None else max_q
    size = lib.dan_window_attention_workspace(N, S, H, Hkv, hd, M, page, window, sinks, chunk, max_q)
    at = [0x1000000000 * (i + 1) for i in range(9)]
    before = ctypes.c_int.in_dll(fake, "launches").value
    st = lib.dan_window_attention(at[0], N, H * hd, at[1], at[2], 5000, page, at[3], M, M, at[4], at[5], S, H, Hkv,
                                  hd, window, sinks, chunk, max_q, 0.1, at[6], at[7], at[8], size, None)
    grids = (ctypes.c_uint * 4 * 64).in_dll(fake, "grids")
    return st, [list(grids[i]) for i in range(before, ctypes.c_int.in_dll(fake, "launches").value)]
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    dan_build.build()
    at = tmp_path_factory.mktemp("fake")
    (at / "fake.c").write_text(FAKE)
    (at / "attr.cpp").write_text(ATTR)
    cuda = os.path.dirname(os.path.dirname(dan_build.nvcc()))
    obj, lib = str(at / "fake.o"), str(at / "libfake.so")
    subprocess.check_call([shutil.which("gcc"), "-fPIC", "-c", str(at / "fake.c"), "-o", obj])
    subprocess.check_call([shutil.which("g++"), "-shared", "-fPIC", "-I", cuda + "/include", obj,
                           str(at / "attr.cpp"), "-o", lib])

    def run(script):
        done = subprocess.run([sys.executable, "-c", PRELUDE + script, lib, ops.LIB_PATH], text=True,
                              capture_output=True, timeout=120)
        assert done.returncode == 0, done.stderr
        return json.loads(done.stdout)

    return run


def threads(launches):
    return [g[2] for g in launches]


def test_kernels_of_a_call(fake):
    """Step kernel with the plan, tile kernel, join; a call of few rows a sequence has no tile
    kernel, one whose keys are never split no join."""
    prompt, few, short = fake("print(json.dumps([attention(), attention(max_q=4), attention(max_q=4, M=2)]))")
    assert prompt[0] == few[0] == short[0] == OK
    assert threads(prompt[1]) == [128, 384, 128] and prompt[1][0][0] == 4 * 8 + 1
    assert threads(few[1]) == [128, 128] and few[1][0][0] == 4 * 8
    assert threads(short[1]) == [128]


@pytest.mark.parametrize("kind,calls", [("ENTRY", 1), ("ENCODE", 5), ("ATTRIBUTES", 1), ("SET", 4)])
def test_a_call_that_cannot_run_whole_launches_nothing(fake, kind, calls):
    """Each of the runtime's answers that a call needs fails once: DAN_ECUDA and no kernel, and
    the next call is as good as any."""
    for n in range(1, calls + 1):
        first, counted, again = fake(f"fail_at[{kind}] = {n}\na = attention()\n"
                                     f"print(json.dumps([a, count[{kind}], attention()]))")
        assert first == [ECUDA, []] and counted == n, n
        assert again[0] == OK and threads(again[1]) == [128, 384, 128], n


def test_no_exception_leaves_a_call(fake):
    """Memory that runs out on the host inside a call: a status, and the next call is as good."""
    first, again = fake("fail_at[SET] = 2\nctypes.c_int.in_dll(fake, 'throws').value = 1\n"
                        "print(json.dumps([attention(), attention()]))")
    assert first == [ECUDA, []]
    assert again[0] == OK and threads(again[1]) == [128, 384, 128]


@pytest.mark.parametrize("registers", [128, 160, 176])
def test_other_register_counts_launch_nothing(fake, registers):
    """The tile kernel's split of its registers needs the count it was written for; calls
    without that kernel are not refused."""
    prompt, few = fake(f"ctypes.c_int.in_dll(fake, 'registers').value = {registers}\n"
                       "print(json.dumps([attention(), attention(max_q=4)]))")
    assert prompt == [ECUDA, []]
    assert few[0] == OK and threads(few[1]) == [128, 128]


REPORT = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_kernel_a' for 'sm_103a'
ptxas info    : Function properties for _kernel_a
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {} registers, used 1 barriers
ptxas info    : Compiling entry function '_kernel_b' for 'sm_103a'
ptxas info    : Function properties for _kernel_b
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {} registers, used 1 barriers
"""


def test_the_build_refuses_other_register_counts():
    src = "dan_attn_tile.cu"
    dan_build.check_registers(src, REPORT.format(168, 168))
    for a, b in ((160, 168), (168, 176)):
        with pytest.raises(RuntimeError, match="registers"):
            dan_build.check_registers(src, REPORT.format(a, b))
    with pytest.raises(RuntimeError, match="no register counts"):
        dan_build.check_registers(src, "")


def test_the_build_asks_for_the_register_counts(monkeypatch, tmp_path):
    """The compile itself: its own source passes, and with another count asked for the
    library is not made."""
    monkeypatch.setattr(dan_build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(dan_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(dan_build, "SOURCES", ["dan_attn_tile.cu"])
    dan_build._compile(False, None)
    os.remove(dan_build.LIB)
    monkeypatch.setattr(dan_build, "REGISTERS", {"dan_attn_tile.cu": 160})
    with pytest.raises(RuntimeError, match="168 registers"):
        dan_build._compile(False, None)
    assert not os.path.exists(dan_build.LIB)
