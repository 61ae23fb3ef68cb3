"""The ABI tests hand fake addresses to the library. Those that expect the device check to stop a
call have to be skipped where there is a device: there the call would launch on them."""
import os
import subprocess
import sys

from conftest import ROOT

PLUGIN = '''
import torch
torch.cuda.is_available = lambda: True


def pytest_collection_finish(session):
    from hadamard_rotated_precision_amd import binding as B

    class Names(dict):
        def __getitem__(self, status):
            assert self.get(status) != "HQ_ERR_DEVICE", "a call passed every check but the device's"
            return dict.__getitem__(self, status)

    B.STATUS_NAMES = Names(B.STATUS_NAMES)
'''


def test_no_call_reaches_the_device_where_there_is_one(tmp_path):
    """Run on the CPU as if there were a GPU: no status is the device check's, and tests ran."""
    (tmp_path / "as_if_there_were_a_gpu.py").write_text(PLUGIN)
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), os.environ.get("PYTHONPATH", "")]),
               HIP_VISIBLE_DEVICES="-1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        "-p", "as_if_there_were_a_gpu", "-m", "not gpu",
                        os.path.join("tests", "test_abi.py"), os.path.join("tests", "test_train_abi.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    print(r.stdout[-3000:] + r.stderr[-2000:])
    assert r.returncode == 0
    tail = r.stdout.strip().splitlines()[-1]
    assert "passed" in tail and "skipped" in tail
