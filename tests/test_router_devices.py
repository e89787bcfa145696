"""What the router's product asks about a device is kept for that device: with a
host-side stand-in for the CUDA runtime, whose two devices run different numbers
of clusters at once. No GPU is touched."""

import ctypes
import shutil
import subprocess
import sys
import textwrap

import pytest

STUB = r"""
#include <string.h>
/* the head of cudaLaunchConfig_t and the attributes of a launch */
struct dim { unsigned x, y, z; };
struct attribute { int id; char pad[4]; union { char pad[64]; struct dim cluster; } val; };
struct config { struct dim grid, block; unsigned long smem; void* stream;
                struct attribute* attrs; unsigned num_attrs; };
int device, failing, launches, grid, cluster, asked;
int cudaGetDevice(int* d) { *d = device; return 0; }
int cudaDeviceGetAttribute(int* v, int what, int d) { *v = 152; return 0; }
int cudaFuncSetAttribute(const void* f, int what, int v) { return 0; }
static unsigned ctas(const struct config* c) {
  for (unsigned i = 0; i < c->num_attrs; ++i)
    if (c->attrs[i].id == 4) return c->attrs[i].val.cluster.x;
  return 1;
}
int cudaOccupancyMaxActiveClusters(int* n, const void* f, const struct config* c) {
  ++asked;
  if (failing) return 999;
  /* device 1 has 16 SMs for clusters of eight, both enough for smaller ones */
  *n = (device == 1 && ctas(c) == 8 ? 16 : 608) / ctas(c);
  return 0;
}
int cudaLaunchKernelExC(const struct config* c, const void* f, void** args) {
  ++launches;
  grid = c->grid.x;
  cluster = ctas(c);
  return 0;
}
"""

CALLS = """
import ctypes, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
L, P, I = ctypes.c_longlong, ctypes.c_void_p, ctypes.c_int
lib.w4a16_router_logits.argtypes = [P, L, P, I, I, I, P, P]
word = lambda name: I.in_dll(stub, name)
for step in sys.argv[3:]:
    word("device").value, word("failing").value = int(step[0]), int(step[1:] == "f")
    word("launches").value = word("grid").value = word("cluster").value = 0
    status = lib.w4a16_router_logits(1 << 20, 256, 1 << 20, 64, 256, 384, 1 << 20, None)
    print(status, *(word(n).value for n in ("launches", "cluster", "grid")))
"""


@pytest.fixture(scope="module")
def calls(tmp_path_factory, lib):
    """calls(*steps): (status, launches, cluster, grid) of the product of 64 rows
    with 384 experts of 256 columns on device "0" or "1", "1f" where the runtime
    cannot say how many clusters run at once; a process of its own each time."""
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    from w4a16_int4_moe_gb300 import build
    at = tmp_path_factory.mktemp("runtime")
    (at / "stub.c").write_text(STUB)
    (at / "calls.py").write_text(textwrap.dedent(CALLS))
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(at / "stub.so"), str(at / "stub.c")],
                   check=True)

    def run(*steps):
        r = subprocess.run([sys.executable, str(at / "calls.py"), str(at / "stub.so"), build.LIB,
                            *steps], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return [tuple(map(int, line.split())) for line in r.stdout.split("\n") if line]
    return run


EIGHTS, FOURS = (0, 1, 8, 48 * 8), (0, 1, 4, 48 * 4)


def test_a_device_does_not_answer_for_another(calls):
    assert calls("0", "1", "0", "1") == [EIGHTS, FOURS, EIGHTS, FOURS]
    assert calls("1", "0", "1") == [FOURS, EIGHTS, FOURS]


def test_no_guess_where_the_runtime_cannot_say(calls):
    from w4a16_int4_moe_gb300 import ops
    failed = (ops.W4A16_ERR_CUDA, 0, 0, 0)
    assert calls("0f", "0", "1f", "1") == [failed, EIGHTS, failed, FOURS]
