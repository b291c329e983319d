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
