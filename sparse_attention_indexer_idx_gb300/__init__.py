"""GB300-native sparse-attention indexer hot path.

libidx.so (CUDA kernels for sm_103a behind a C ABI, include/idx.h) computes the
DSA indexer score and its exact top-K, DoSA safe-upper-bound pruning, the
segment-witness covering merge, MiniMax block-max selection, decode attention
over a shared prefix and private caches or selected slots, and eviction from
the caches by attention mass.  `binding` is the thin ctypes layer over it;
`serving` runs a decode step's operators together; `workloads` makes seeded
synthetic inputs.
"""
