"""Rules that every kernel source keeps and that a run would show only by
chance (no GPU): what may hang or read too early is checked where it is written."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "flow_matching_dit_cosmot_b200", "csrc")


def source(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


FILES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")))


@pytest.mark.parametrize("name", FILES)
def test_no_drain_gives_up_for_a_failure_of_others(name):
    """The wait for a CTA's own copies and products in flight ends when they have landed or after its time limit,
    never because the status word holds something: mbar_wait (and warp_wait over it) returns at once then."""
    assert not re.search(r"\b(mbar_wait|warp_wait)\([^;]*Drain\)", source(name))


def test_warps_converge_before_an_aligned_cluster_barrier():
    """barrier.cluster .aligned wants every lane of the warp at the same instruction; it is issued from one place, which
    brings them together first."""
    with open(os.path.join(CSRC, "ptx.cuh"), encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert text.count("barrier.cluster.arrive") == 1
    assert re.search(r"void cluster_sync\(\) \{\s*__syncwarp\(\);\s*asm volatile\(\s*\"barrier\.cluster\.arrive", text)
    for name in FILES:
        assert "barrier.cluster" not in source(name)


# What kernels that are launched early may hold to be constant while they live: weights, and the tables that only
# kernels which never trigger their successor write.
CONSTANTS = {"g", "g0", "g1", "gv", "w_in", "w_out", "cs", "cs_row", "t", "p.chunk"}
WRITTEN_ONLY = {"rmsnorm_f32in_kernel": "out", "rmsnorm_block_kernel": "out", "rmsnorm_kernel": "out", "action_embed_kernel": "h"}


@pytest.mark.parametrize("name", FILES)
def test_no_load_of_an_earlier_kernels_output_may_pass_the_wait_for_it(name):
    """__ldg and __restrict__ let the compiler lift a load above griddepcontrol.wait, where the kernel before still
    writes.  Kernels without that wait may use them."""
    text = re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", source(name))
    for m in re.finditer(r"__ldg\((?:reinterpret_cast<[^>]*>\()?\s*([\w.]+)", text):
        assert m.group(1) in CONSTANTS, f"__ldg of {m.group(1)}"
    heads = list(re.finditer(r"(?:__global__|__device__ __forceinline__)[^;{(]*?(\w+)\(([^{;]*)\)\s*\{", text))
    waits = {m.group(1): "pdl_wait();" in text[m.end():m.end() + 1600] for m in heads}
    for m in heads:
        if not waits[m.group(1)] and m.group(0).startswith("__global__"):
            continue
        for const, var in re.findall(r"(const )?\w+\s*\*\s*__restrict__\s+(\w+)", m.group(2)):
            if const:
                assert var in CONSTANTS, f"{m.group(1)}: {var} is read"
            else:
                assert WRITTEN_ONLY.get(m.group(1)) == var, f"{m.group(1)}: {var} may be read"


# Places that write global memory in the 8-bit cache's kernels, and how many of them the debug build checks: every one
# whose index is not the thread's own loop variable below its extent.
KV8_CHECKS = {"store_kernel": 2, "evict_select_kernel": 2, "evict_move_kernel": 2, "tile_attention_kernel": 1, "tile_join_kernel": 1,
              "tile_weigh_kernel": 1, "rows_attention_kernel": 3, "rows_join_kernel": 1, "rows_weigh_kernel": 1}


def test_the_debug_build_checks_every_store_of_the_8_bit_cache():
    seen = {}
    for name in [f for f in FILES if f.startswith("kv8")]:
        text = re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", source(name))
        parts = re.split(r"__global__[^;{(]*?(\w+)\(", text)
        for kernel, body in zip(parts[1::2], parts[2::2]):
            seen[kernel] = body.split("\n}\n")[0].count("dcheck(")
    assert seen == KV8_CHECKS
