"""A run of several GPUs uses no cluster that loads by multicast (clusters of two pairs)."""
import os
import subprocess
import sys

import pytest
import torch

from tests._gpu import built

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import rag_non_prefix_gb300 as cb, torch
torch.cuda.init()
shapes = [(m, n, k, e) for m in (192, 535, 1357, 8320) for n, k in ((4096, 4096), (7168, 20480), (28672, 4096)) for e in (0, 1, 2)]
for pairing in (0, 2, 4):
    cb.cb_gemm_set_pairing(pairing)
    print(*(sum(f"cluster={cl}" in cb.cb_gemm_describe(*s) for s in shapes) for cl in (2, 4)))
"""


@pytest.mark.parametrize("env,multicast", [({}, True), ({"WORLD_SIZE": "1"}, True), ({"WORLD_SIZE": "2", "RANK": "0"}, False),
                                           ({"WORLD_SIZE": "8", "RANK": "3"}, False)])
def test_clusters_of_two_pairs_only_in_runs_of_one_gpu(env, multicast):
    built()
    multicast = multicast and torch.cuda.device_count() == 1
    base = {k: v for k, v in os.environ.items() if k not in ("WORLD_SIZE", "RANK", "LOCAL_RANK")}
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, env={**base, **env}, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    (_, auto4), (pairs, _), (_, two_pairs) = (map(int, line.split()) for line in r.stdout.strip().splitlines())
    assert pairs == 36
    assert two_pairs == 36 if multicast else (auto4, two_pairs) == (0, 0)
