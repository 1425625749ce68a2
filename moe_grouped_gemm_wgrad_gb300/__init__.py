"""Grouped MoE GEMMs for GB300 (sm_103a): MXFP8 quantize, MXFP8 grouped wgrad, fp32 and
MXFP8 grouped dgrad, the MXFP8 forward, and the routed layer around them (router, row
tables, fused epilogues, combine), as a C-ABI CUDA library (``libmgw.so``) with a thin
ctypes binding (:mod:`moe_grouped_gemm_wgrad_gb300.mgw`).

Importing this package loads nothing; the library is loaded on first use and a
missing or unbuilt library raises instead of falling back to anything else.
"""
