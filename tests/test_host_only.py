"""The argument-check modules hand the library made-up device addresses; some
of their calls pass every host check and end only because no device is there.
Where a GPU is visible none of them may run."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_made_up_addresses_stay_off_a_visible_gpu(tmp_path):
    # a stand-in for the GPU: the count alone (nothing here can reach one)
    (tmp_path / "one_gpu.py").write_text("import torch\ntorch.cuda.device_count = lambda: 1\n")
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT]),
               HIP_VISIBLE_DEVICES="-1")
    args = [sys.executable, "-m", "pytest", "-q", "-p", "one_gpu", "-p", "no:cacheprovider"]
    files = [os.path.join("tests", f) for f in ("test_abi.py", "test_abi_layer.py")]
    p = subprocess.run(args + files, cwd=ROOT, env=env, capture_output=True, text=True)
    last = p.stdout.strip().splitlines()[-1]
    assert p.returncode == 0 and "skipped" in last and "passed" not in last, p.stdout[-2000:]
    # a module without such addresses runs as before
    p = subprocess.run(args + [os.path.join("tests", "test_oracle_layer.py")], cwd=ROOT, env=env,
                       capture_output=True, text=True)
    last = p.stdout.strip().splitlines()[-1]
    assert p.returncode == 0 and "passed" in last and "skipped" not in last, p.stdout[-2000:]
