"""The sort by expert in a process of its own: what a launch asks for goes by its
own number of experts, not by what an earlier call has asked for."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (Growing numbers of experts around 48 KB of tables, the most that a launch has
# without asking; more choices than are placed without a sort.)
CHILD = """
import torch
import fp32_sgemm_gb300 as sg
for G in (1, 352, 353, 358, 359, 360, 361, 362, 1024, 360):
    T, k = 4100, 2
    g = torch.Generator(device="cuda").manual_seed(G)
    experts = torch.randint(-1, G + 1, (T, k), generator=g, device="cuda")
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None]
    rows, slots, ends = sg.expert_dispatch(x, experts, G)
    flat = experts.reshape(-1)
    key = torch.where((flat >= 0) & (flat < G), flat, G)
    order = torch.argsort(key, stable=True)
    want = torch.empty_like(order)
    want[order] = torch.arange(T * k, device="cuda")
    assert torch.equal(slots.reshape(-1).long(), torch.where(key < G, want, -1 - want)), G
    assert torch.equal(ends.long(), torch.bincount(key, minlength=G + 1)[:G].cumsum(0)), G
    assert torch.equal(rows[:, 0], torch.where(key[order] < G, (order // k).float(), 0.0)), G
print("sorted")
"""


def test_any_number_of_experts_comes_first():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    done = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.endswith("sorted\n"), done.stderr
