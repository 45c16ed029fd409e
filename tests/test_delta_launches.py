"""Launches of the gated delta rule, with the runtime's launch call replaced by one that records and
fails where it is told to (CPU, a process of its own): a launch that fails is the call's status,
whatever follows it, and every grid keeps to the runtime's limit."""
import json
import os
import subprocess
import sys

import pytest

import state_space_model_amd as ssd
import test_gpu_delta_chains
import test_gpu_delta_pairs
import test_gpu_delta_terms as terms

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, UNSUP, HIP = 0, 5, 7

SHIM = r"""
#include <stdint.h>
#include <stddef.h>
typedef struct { uint32_t x, y, z; } dim;
int shim_count, shim_fail, shim_sticky, shim_last;
uint32_t shim_sizes[64][2];
static dim grid, block;
int __hipPushCallConfiguration(dim g, dim b, size_t lds, void* stream) { grid = g; block = b; return 0; }
int __hipPopCallConfiguration(dim* g, dim* b, size_t* lds, void** stream) {
  *g = grid; *b = block; *lds = 0; *stream = 0;
  return 0;
}
int hipLaunchKernel(const void* f, dim g, dim b, void** args, size_t lds, void* stream) {
  const int bad = shim_count == shim_fail ? 719 : 0;
  if (shim_count < 64) { shim_sizes[shim_count][0] = g.x; shim_sizes[shim_count][1] = b.x; }
  ++shim_count;
  if (bad || !shim_sticky) shim_last = bad;   /* the error stays until it is read, or until the next launch */
  return bad;
}
int hipGetLastError(void) { const int e = shim_last; shim_last = 0; return e; }
"""

CHILD = r"""
import ctypes, json, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
N = lambda n: ctypes.c_int.in_dll(shim, "shim_" + n)
class Desc(ctypes.Structure):
    _fields_ = ([(f"i{i}", ctypes.c_int64) for i in range(12)] + [(f"j{i}", ctypes.c_int32) for i in range(4)]
                + [(f"f{i}", ctypes.c_float) for i in range(4)])
for fn, n in (("ssd_delta_scan_workspace_bytes", 0), ("ssd_delta_scan_backward_workspace_bytes", 0)):
    getattr(lib, fn).restype = ctypes.c_size_t
at = lambda i: ctypes.c_void_p((1 << 45) + (i << 42))      # never read: nothing is launched
out = []
for name, io, Bt, T, H, G, P, K in json.loads(sys.argv[3]):
    d = Desc(Bt, T, H, P, K, G, G * K, G * K, H * P, G * K, G * K, H * P, io, 1, 1, 1, 0.0, float("inf"), 1e-6, 1.0)
    r = ctypes.byref(d)
    def run():
        if name == "step":
            return lib.ssd_delta_step(r, *[at(i) for i in range(9)], None)
        pointers = 11 if name == "scan" else 19
        need = getattr(lib, "ssd_delta_scan_workspace_bytes" if name == "scan" else
                       "ssd_delta_scan_backward_workspace_bytes")(r)
        call = lib.ssd_delta_scan if name == "scan" else lib.ssd_delta_scan_backward
        return call(r, *[at(i) for i in range(pointers)], ctypes.c_size_t(need), None)
    N("fail").value, N("count").value, N("last").value, N("sticky").value = -1, 0, 0, 1
    status = run()
    launches = N("count").value
    sizes = ((ctypes.c_uint32 * 2) * 64).in_dll(shim, "shim_sizes")
    grids = [list(sizes[i]) for i in range(launches)]
    failed = []
    for sticky in (0, 1):
        for i in range(launches):
            N("fail").value, N("count").value, N("last").value, N("sticky").value = i, 0, 0, sticky
            failed.append([run(), N("count").value])
    out.append([status, grids, failed])
print(json.dumps(out))
"""

# rows, tokens, heads, groups, values, keys
SHAPES = [(1, 70, 4, 2, 24, 40), (3, 130, 32, 8, 40, 128), (3, 130, 16, 16, 40, 72), (5, 65, 32, 8, 64, 64),
          (2, 64, 80, 80, 64, 128)]
CALLS = [(name, io, *s) for name in ("scan", "back", "step") for io in (0, 1) for s in SHAPES]


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    at = tmp_path_factory.mktemp("launches")
    src, so = at / "shim.c", at / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)

    def ask(calls):
        lib = os.path.join(os.path.dirname(ssd.__file__), "libssd.so")
        r = subprocess.run([sys.executable, "-c", CHILD, str(so), lib, json.dumps(calls)], capture_output=True,
                           text=True, cwd=ROOT)
        assert r.returncode == 0, r.stderr[-2000:]
        return json.loads(r.stdout)

    return ask


def test_a_failed_launch_is_the_status(answers):
    for call, (status, grids, failed) in zip(CALLS, answers(CALLS)):
        name, io, Bt, T, H, G, P, K = call
        assert status == OK and len(grids) == {"scan": 2, "step": 1, "back": 4 + (H != G)}[name], call
        for i, (code, count) in enumerate(failed):
            assert code == HIP, (call, i)
            assert count == i % len(grids) + 1, (call, i)     # nothing reads what a failed launch did not write


# the largest sizes: rows of the keys' gradients up to 2^27 - 8 (eight to a workgroup of 256 threads,
# and threads count in 32 bits), workgroups below 2^24
LARGE = [("back", 0, 1, 22369621, 6, 3, 8, 128, UNSUP), ("back", 1, 1, 22369621, 6, 3, 8, 72, UNSUP),
         ("back", 1, 1, 33554431, 4, 2, 8, 128, UNSUP), ("back", 1, 1, 33554430, 4, 2, 8, 128, OK),
         ("back", 0, 1, 33554430, 4, 2, 8, 64, OK), ("scan", 1, 1, 64 * 4194303, 4, 4, 256, 128, OK),
         ("scan", 0, 4194303, 64, 4, 1, 16, 128, OK), ("step", 1, 4194303, 1, 4, 1, 16, 128, OK),
         ("step", 0, 8191, 1, 256, 1, 128, 128, OK)]


def test_grids_keep_to_the_limit(answers):
    for call, (status, grids, failed) in zip(LARGE, answers([c[:-1] for c in LARGE])):
        assert status == call[-1], (call, status)
        assert bool(grids) == (status == OK), call
        for groups, threads in grids:
            assert 0 < groups * threads < 1 << 32, (call, groups, threads)


def test_every_kind_of_chain_is_tested(answers):
    """The launches of the GPU tests' sizes: a workgroup of 256 threads to 16 value columns, of 512 to
    32, or of 256 to 64 (bfloat16)."""
    kinds = {"alone": (256, 16), "pairs": (512, 32), "owned": (256, 64)}
    asked = [("back", s, k) for k, shapes in (("alone", terms.ALONE), ("pairs", terms.PAIRS), ("owned", terms.OWNED))
             for s in shapes]
    for (Bt, H, G, P), back in zip(test_gpu_delta_chains.KINDS + test_gpu_delta_pairs.KINDS,
                                   ("alone", "owned", "owned", "pairs", "pairs")):
        asked.append(("back", (Bt, 130, H, G, P, 40), back))
    for (Bt, H, G, P), scan in zip(test_gpu_delta_chains.KINDS, ("alone", "pairs", "owned")):
        asked.append(("scan", (Bt, 130, H, G, P, 40), scan))
    for (name, shape, kind), (_, grids, _) in zip(asked, answers([(n, 1, *s) for n, s, _ in asked])):
        Bt, T, H, G, P, N = shape
        threads, columns = kinds[kind]
        ways = 2 if name == "back" else 1
        assert grids[1] == [ways * Bt * H * ((P + columns - 1) // columns), threads], (name, shape, kind)
