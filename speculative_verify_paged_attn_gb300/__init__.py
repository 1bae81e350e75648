"""GB300-native paged speculative verification: paged_verify_attn, spec_accept,
spec_accept_tree and block_table_commit behind a C ABI (libsvpa.so), with the
admission of prompts (block_table_build, kv_write, paged_prompt_attn), verification
behind a shared prefix (prefix_verify_attn) and logits_process.

``svpa`` is the ctypes binding (argument marshalling only); ``workloads`` draws
seeded synthetic inputs.
"""
