"""No kernel loads through TMA multicast. The benchmark runs every workload of
its list on each rank of a job of any number of GPUs, and a library call cannot
see how many GPUs the job that it belongs to has, so the copies that a cluster's
CTAs need are each CTA's own."""
import glob
import os
import re

import bench
from mla_latent_kv_cache_gb300 import build as mbuild


def _code(path):
    """A source file without its comments."""
    text = open(path).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_kernel_source_names_a_multicast_copy():
    files = sorted(f for pat in ("*.cu", "*.cuh", "*.inc") for f in glob.glob(os.path.join(mbuild.CSRC, pat)))
    assert {os.path.basename(f) for f in files} >= set(mbuild.SOURCES)  # everything that is built is looked at
    for f in files:
        assert "multicast" not in _code(f), f


def test_the_workload_with_128_query_rows_runs_on_every_rank():
    # the one whose row groups once shared their tiles by multicast: on the default list of any --gpus N
    assert "verify8" in bench.SIDE_WORKLOADS and "verify8" in bench.CONFIG_TEXT
    assert int(bench.verify_qlens(128, qmax=8).max()) * 16 == 128
