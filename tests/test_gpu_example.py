"""The decoder example: the cached path gives what the prompt path gives."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prompt,samples,steps", [(1024, 8, 8), (37, 3, 70), (64, 1, 2)])
def test_decoder_example(dtype, prompt, samples, steps):
    cmd = [sys.executable, os.path.join(ROOT, "examples", "decoder_block.py"), "--prompt", str(prompt), "--samples",
           str(samples), "--steps", str(steps), "--dtype", dtype]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    # pages after half of the samples ended: the shared ones and the other samples' own
    full = prompt // 64
    own = -(-(prompt + steps) // 64) - full
    kept = samples // 2
    live = full + kept * own if kept else 0
    assert f"half of the samples ended: {live}, " in r.stdout, r.stdout
