"""The base projection's line of the bench runs on one GPU only: its kernel loads with cluster multicast,
which is kept to processes that have the GPU to themselves.  On the CPU; nothing is launched."""

import json

import pytest
import torch

import bench


def test_the_base_line_refuses_more_than_one_gpu():
    with pytest.raises(SystemExit, match="one GPU"):
        bench.run_base_line(10, 3, 0.0, 2, 0, 0)
    with pytest.raises(SystemExit, match="one GPU"):
        bench.head_line("base_fused", bench.parse_args(["--workload", "base_fused"]), 2, 0, 0)


@pytest.mark.parametrize("world", [1, 2])
def test_the_other_lines_run_without_it(monkeypatch, capsys, world):
    ran = []

    def line(name):
        def run(*a):
            ran.append(name)
            return {"value": 1.0, "ms_per_step": 1.0, "gpu_launches": 1}
        return run

    monkeypatch.setattr(bench, "dist_info", lambda: (world, 0, 0))
    monkeypatch.setattr(torch.cuda, "set_device", lambda d: None)
    monkeypatch.setattr(torch.distributed, "init_process_group", lambda **kw: None)
    monkeypatch.setattr(torch.distributed, "destroy_process_group", lambda: None)
    for name in ("config_line", "run_backward_line", "run_base_line", "head_line"):
        monkeypatch.setattr(bench, name, line(name))
    assert bench.main(["--cpu-seconds", "0"]) == 0
    assert ran.count("run_base_line") == (1 if world == 1 else 0)
    out = json.loads(capsys.readouterr().out)
    assert "backward" in out["per_config"] and ("base_fused" in out["per_config"]) == (world == 1)
