"""Which tile a forced plan kind gives the block operators, and which kinds they
do not have and leave to their own choice (CPU only: plan queries)."""
import pytest

import nvfp4_block_scaled_07_amd as nv

EPILOGUE = {9: "tile64x64k4", 10: "kreg16x16k8", 11: "kreg32x16k8", 12: "kreg32x32k8", 14: "tile256x256w8k256_mfma32",
            15: "tile128x128k256_mfma32", 16: "tile256x192w8k256_mfma32", 32: "kreg16x32k8", 34: "tile64x64k4w8"}
GATED = {9: "gated64x32k4", 10: "gatedreg16x16k8", 12: "gatedreg32x16k8", 14: "gated256x128w8", 15: "gated128x64",
         32: "gatedreg16x32k8", 33: "gatedreg16x8k8"}
SHAPES = [(70, 270, 1536), (257, 195, 768), (1, 2048, 6144), (4096, 4096, 512)]


@pytest.mark.parametrize("query,kinds", [(nv.nvfp4_gemm_epilogue_plan, EPILOGUE), (nv.nvfp4_gemm_gated_plan, GATED)])
@pytest.mark.parametrize("shape", SHAPES)
def test_forced_kinds(query, kinds, shape, force_plan):
    own = query(*shape)
    assert own in kinds.values()
    for kind in range(40):
        force_plan(nv.FAMILY_GEMM, kind)
        assert query(*shape) == kinds.get(kind, own), kind
    force_plan(nv.FAMILY_GEMM, -1)
    assert query(*shape) == own
