"""The key of the committed DRAM counters follows the matmuls' sources, and no others."""
import os
import shutil

import bench

CSRC = os.path.join(bench.ROOT, "weight_only_int4_02_gb300", "csrc")


def digest_with(tmp_path, name):
    """The digest of a copy of the sources in which one file has another line of code."""
    copy = str(tmp_path / name)
    shutil.copytree(CSRC, copy)
    with open(os.path.join(copy, name), "a") as f:
        f.write("\nstatic int one_more_line;\n")
    return bench.source_digest(copy)


def test_the_digest_follows_the_matmuls_sources(tmp_path):
    now = bench.source_digest()
    assert bench.source_digest(CSRC) == now
    for name in ("api.cu", "decode.cu", "decode.cuh", "gemm_tc.cuh", "gemm_tc128.cu", "gemv.cu", "pack.cu", "ptx.cuh"):
        assert digest_with(tmp_path, name) != now, name


def test_the_serving_steps_sources_leave_it_as_it_is(tmp_path):
    now = bench.source_digest()
    for name in ("api_serve.cu", "binding.cpp", "kv4.cuh", "kv4_attn.cu", "kv4_cache.cu", "kv4_prompt.cu", "launch.cuh", "sample.cu",
                 "sample.cuh"):
        assert digest_with(tmp_path, name) == now, name
