"""Modulated deformable 2-D convolution (DCNv2) for MI355X (gfx950), and
attention over the maps it produces.

The computation lives in libmdcn.so (C ABI in include/mdcn.h, HIP kernels in
csrc/); ``mdcn`` is its Python binding, ``attention`` that of the attention
operators with ``map_attention`` as their example, and ``workloads`` draws
seeded synthetic inputs.  Importing the package loads nothing.
"""
