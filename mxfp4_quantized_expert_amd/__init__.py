"""MI355X-native MXFP4 mixture-of-experts expert FFN (gfx950 HIP kernels behind a C ABI).

Submodules:
  binding   -- binding of libmxfp4moe.so (mxfp4_dequantize, moe_mxfp4_route,
               moe_mxfp4_forward, and the layer's separate operators with their
               gradients: moe_permute, moe_unpermute, moe_route_backward,
               moe_mxfp4_linear, moe_nvfp4_linear, and around the experts
               moe_rms_norm, moe_fp8_quantize, moe_fp8_linear, moe_swiglu,
               moe_balance_loss); argument marshalling only.
  workloads -- seeded synthetic layers (inputs only, no arithmetic of the method).

Importing the package loads nothing; ``binding.load()`` loads the HIP library
and raises if it has not been built.
"""

__all__ = ["binding", "workloads"]
