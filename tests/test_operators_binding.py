"""The binding's C module by itself (no GPU)."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

import __graft_entry__ as entry
from speculative_state_replay_gb300 import _lib, build

FUNCTIONS = ("rssm_delta_step", "rssm_delta_prefill", "rssm_verify", "rssm_gated_norm", "rssm_residual_norm")


@pytest.fixture(scope="module", autouse=True)
def _built():
    entry.build()


def test_module_carries_its_interpreter():
    """Another interpreter, or another release of this one, does not import this one's build."""
    assert os.path.basename(_lib.fast().__file__) == "_call" + sysconfig.get_config_var("EXT_SUFFIX")


def test_one_library(tmp_path):
    """A library loaded from elsewhere is the one that the C module calls."""
    other = str(tmp_path / "other.so")
    shutil.copy(_lib.LIB_PATH, other)
    code = ("import sys; from speculative_state_replay_gb300 import _lib; _lib.load(sys.argv[1]); _lib.fast();"
            "print(*{l.split()[-1] for l in open('/proc/self/maps') if l.rstrip().endswith(('other.so', 'librssm.so'))})")
    r = subprocess.run([sys.executable, "-c", code, other], capture_output=True, text=True, cwd=build.ROOT, check=True)
    assert r.stdout.split() == [other]


def test_other_threads_run_meanwhile(tmp_path):
    """A call that takes long -- a launch into a full queue -- stops no other Python thread: the module linked to a
    library whose calls take 0.2 s."""
    stub = tmp_path / "stub.c"
    stub.write_text("#include <unistd.h>\n" + "".join(f"int {f}() {{ usleep(200000); return 7; }}\n" for f in FUNCTIONS))
    lib = tmp_path / "librssm.so"
    module = tmp_path / ("_call" + sysconfig.get_config_var("EXT_SUFFIX"))
    subprocess.run(["gcc", "-shared", "-fPIC", str(stub), "-o", str(lib)], check=True)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(build.ROOT, "include"),
                    build.CALL_SRC, "-o", str(module), str(lib), "-Wl,-rpath,$ORIGIN"], check=True)
    code = """
import sys, threading, time
sys.path.insert(0, sys.argv[1])
import _call
args = dict(rssm_delta_step=[0]*9 + [1.0] + [0]*11, rssm_delta_prefill=[0]*9 + [1.0] + [0]*10, rssm_verify=[0]*17,
            rssm_gated_norm=[0]*10 + [1e-5] + [0]*4, rssm_residual_norm=[0]*8 + [1.0] + [0]*3 + [1e-5] + [0]*5)
for name, a in args.items():
    ticks, stop = [], threading.Event()
    def tick():
        while not stop.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.005)
    t = threading.Thread(target=tick)
    t.start()
    time.sleep(0.02)
    t0 = time.monotonic()
    status = getattr(_call, name)(*a)
    t1 = time.monotonic()
    stop.set()
    t.join()
    print(name, status, t1 - t0 > 0.19, sum(t0 + 0.01 < x < t1 - 0.01 for x in ticks) > 3)
"""
    r = subprocess.run([sys.executable, "-c", code, str(tmp_path)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert r.stdout.splitlines() == [f"{f} 7 True True" for f in FUNCTIONS]


def test_low_parts_of_the_sums():
    """pend_cl may be missing; what is given is checked like pend_c."""
    import ctypes

    lib, at = _lib.load(), 1 << 20
    c = _lib.RssmDeltaCacheStruct(num_slots=4, nkheads=2, nvheads=4, dkey=128, dvalue=64, npredicted=4, state_dtype=0, state=at,
                                  state_slot_stride=4 * 64 * 128, pend_k=at, pend_k_slot_stride=2 * 2 * 4 * 128, pend_w=at,
                                  pend_w_slot_stride=2 * 4 * 4 * 64, pend_c=at, pend_c_slot_stride=2 * 4 * 4, pend=at, error_word=at)
    assert lib.rssm_delta_scratch_bytes(ctypes.byref(c), 1, 1) > 0
    for pointer, stride, ok in ((at, 32, True), (at + 4, 40, True), (at + 2, 32, False), (at, 31, False), (at, -32, False)):
        c.pend_cl, c.pend_cl_slot_stride = pointer, stride
        assert (lib.rssm_delta_scratch_bytes(ctypes.byref(c), 1, 1) > 0) == ok
