"""The DRAM traffic that bench.py reports with a kernel's time is taken from
profiles/traffic.json while the kernel's sources are those it was captured on.
After a change to them the capture is repeated as profiles/dram_traffic_per_launch.md
says; until then the bench reports none."""
import json
import os

import bench


def test_captured_traffic_belongs_to_the_current_sources():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        figures = json.load(f)
    old = [(workload, phase) for workload, phases in figures.items() if not workload.startswith("_")
           for phase in phases if bench.ncu_traffic(phase, workload) is None]
    assert old == []
